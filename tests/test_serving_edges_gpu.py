"""The serving operators on the GPU at the ends of their ranges: gates whose
SwiGLU factors leave float32 though the product does not."""
import numpy as np
import pytest

import serving_ref as ref
from helpers import to_device
from test_serving_gpu import T, check_codes, offsets_of, sync, tre   # noqa: F401 (tre: the fixture)

pytestmark = pytest.mark.gpu


# (gate, up): below -88.73 the definition's denominator 1 + e^-g passes float32's range and the result is a zero;
# between, and far above, the result is an ordinary number although g * u or 1 / (1 + e^-g) alone is not.
GATES = [(-20.0, 1e38), (-60.0, -3e38), (-86.0, 1e37), (-87.0, 1e38), (-87.4, -1e38), (-88.0, 1e38), (-88.7, 1e38),
         (-88.8, 1.0), (-89.0, 1e38), (-100.0, 1e30), (-150.0, -1.0), (-1e4, 1e38), (-1e20, 1e20), (-3e38, 3e38),
         (-3e38, 1.0), (-1.0, 1e38), (-1e-30, 1e38), (0.0, 1e38), (1e-30, -1e38), (1.0, 3e37), (20.0, 1e37),
         (89.0, 1e36), (1e20, 1e18), (3e38, 1.0), (3e38, 1e-30)]


@pytest.mark.parametrize("rows", [10, 40, 80, 160])   # tiles of 32 and 64 rows (bf16 inside), 128 and 288 (8 bits)
def test_gate_up_extreme_gates(tre, rows):
    """Finite gates and ups whose silu(gate) * up is finite never give NaN codes, and give that product."""
    torch = T()
    E, d, I = 32, 512, 1024                            # 8 column tiles an expert: a tile for every compute unit
    g, u = (np.resize(np.array(v, np.float32), E * rows).astype(np.float64) for v in zip(*GATES))
    # row r's gate comes from its first k and its first scale, its up from the second block of k and that scale
    x = torch.zeros((E * rows, d))
    x[:, 0], x[:, 128] = torch.from_numpy(np.sign(g)), torch.from_numpy(np.sign(u))
    xs = np.ones((E * rows, 4), np.float32)
    xs[:, 0], xs[:, 1] = np.abs(g), np.abs(u)
    w = torch.zeros((E, 2 * I, d))
    w[:, :I, 0] = 1.0
    w[:, I:, 128] = torch.tensor([1.0, 0.5, -1.0, 0.25]).repeat(I // 4)
    f8 = torch.float8_e4m3fn
    hq, hs = tre.moe_gate_up_swiglu_fp8(x.to(f8).cuda(), to_device(xs), offsets_of([rows] * E), w.to(f8).cuda(),
                                        torch.ones((E, 2, I // 128, d // 128), device="cuda"))
    sync()
    ups = u[:, None] * np.resize([1.0, 0.5, -1.0, 0.25], I)
    with np.errstate(over="ignore"):
        silu = (g / (1.0 + np.exp(-g)))[:, None]
    h = silu * ups
    # exponential, its correction, sum, reciprocal and two products: 8 half steps; 1e-37 covers results below
    # float32's normal range; where the denominator passes it, |silu| <= 88.73 e^-88.73 = 2.7e-37 may become zero
    bound = 8 * ref.HALF_F32 * np.abs(h) + 1e-37 + np.where(g < -88.72, 2.7e-37, 0.0)[:, None] * np.abs(ups)
    check_codes(hq, hs, h, bound, f"{rows} rows an expert")
