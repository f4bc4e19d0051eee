"""The training operators' bf16 products in calls of several tiles a workgroup:
the stream of stages that runs on across an epilogue, tall tiles behind tall tiles,
tiles that are claimed, and last tiles that are cut into pieces; bit for bit where
every sum is exact (in 16-bit codes within their bound).

Each case asserts that its products have the tiles it is there for."""
import numpy as np
import pytest

import training_exact as exact
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu



MEAN = {"256": 1500, "tall": 268, "128": 100, "64": 40}     # rows of an expert, by the tiles that they lead to


def counts_of(kind, E):
    """E counts around the kind's mean, an empty expert and a tall tile's edges among them."""
    n = np.random.default_rng(E).integers(MEAN[kind] * 7 // 8, MEAN[kind] * 9 // 8, E)
    edges = [0, 1, 255, 256, 257, 288, 289]
    n[1:1 + min(len(edges), E // 4)] = edges[:min(len(edges), E // 4)]
    return [int(v) for v in n]


def row_tiles(kind, counts):
    if kind != "tall":
        return sum(-(-n // int(kind)) for n in counts)
    full = [-(-n // 256) for n in counts]
    return sum(m - (1 if m > 1 and n - 256 * (m - 1) <= 32 else 0) for m, n in zip(full, counts))


def rounds(kind, counts, columns):
    """Tiles of a product with that many columns of 256 (gate/up: 128 of I), by the places for them."""
    import torch
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    per_cu = 2 if kind in ("128", "64") else 1
    return row_tiles(kind, counts) * columns / (cus * per_cu)


def right_kind(kind, counts):
    R, E = sum(counts) + exact.EXTRA, len(counts)
    return {"256": R > 384 * E, "tall": 128 * E <= R <= 288 * E, "128": 64 * E < R < 128 * E,
            "64": R <= 64 * E and E <= 128}[kind]


# (kind, experts, d, I): a wide I has many tiles in gate/up and the SwiGLU backward, a wide d in down and dx
CASES = [("256", 16, 256, 2048), ("256", 24, 2048, 320), ("tall", 120, 256, 1088), ("tall", 120, 1088, 256),
         ("128", 128, 256, 2048), ("128", 128, 2048, 256), ("64", 128, 256, 2112), ("64", 128, 2112, 256)]


@pytest.mark.parametrize("kind,E,d,I", CASES)
def test_forward(tre, kind, E, d, I):
    counts = counts_of(kind, E)
    assert right_kind(kind, counts)
    assert max(rounds(kind, counts, -(-I // 128)), rounds(kind, counts, -(-d // 256))) > 1.5
    if kind in ("256", "tall") and I > d:
        assert rounds(kind, counts, -(-I // 128)) >= 4       # claimed tiles: gate/up is d / 32 = 8 stages deep
    exact.check_forward(tre, counts, d, I)


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("kind,E,d,I", CASES)
def test_backward(tre, kind, E, d, I, again):
    counts = counts_of(kind, E)
    assert right_kind(kind, counts)
    assert max(rounds(kind, counts, -(-I // 256)), rounds(kind, counts, -(-d // 256))) > 1.5
    exact.check_backward(tre, counts, d, I, again)


def pairs_of(counts, k, seed):
    """[T, k] pairs that give every expert its count, the last tokens' filled with -1."""
    idx = np.repeat(np.arange(len(counts)), counts)
    idx = np.concatenate([idx, np.full(-len(idx) % k + 3 * k, -1)])
    np.random.default_rng(seed).shuffle(idx)
    return idx.reshape(-1, k).astype(np.int32)


@pytest.mark.parametrize("kind,E,d,I", CASES)
def test_layer(tre, kind, E, d, I):
    counts = counts_of(kind, E)
    assert right_kind(kind, counts)
    assert exact.check_layer(tre, pairs_of(counts, 2, E), d, E, I) == counts


# (rows of each expert, d, I): y's tiles pass whole rounds of 256 by at most half a round, and I is deep enough for two
# pieces or more of each (layers: float32 rows, summed by themselves; grouped rows: bf16)
TAILS = {"256": ([1536] * 5 + [1024, 0, 1500], 2048, 1024), "tall": ([270, 256, 288, 100] * 9, 2048, 1024)}


@pytest.mark.parametrize("kind", list(TAILS))
def test_split_tails(tre, kind):
    counts, d, I = TAILS[kind]
    assert right_kind(kind, counts)
    over = rounds(kind, counts, d // 256)
    assert over > 1 and 0 < over % 1 <= 0.5
    exact.check_forward(tre, counts, d, I)
    assert exact.check_layer(tre, pairs_of(counts, 2, 5), d, len(counts), I) == counts


def test_claimed_tiles_of_float32_rows(tre):
    """Four rounds of the layer's y in tiles of 256 rows and in tall ones, 16 stages deep."""
    for kind, E in (("256", 28), ("tall", 128)):
        counts, d, I = counts_of(kind, E), 2048, 512
        assert right_kind(kind, counts) and rounds(kind, counts, d // 256) >= 4
        assert exact.check_layer(tre, pairs_of(counts, 2, 6), d, E, I) == counts
