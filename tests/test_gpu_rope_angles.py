"""The angles of pa_rope_append: cosine and sine themselves, by turning (1, 0) in fp32, against exact arithmetic.

Tolerance: sincospif is off by at most 1 ulp (a relative 2^-23).  What its fp32 argument leaves of the angle, d, at
most pi 2^-25, is rounded twice and multiplied by pi as a float (2.5 x 2^-24 in all) and by a value that is off by
2^-23: below (2.5 + 2) 2^-24 pi 2^-25 < 2^-45.  The sum is rounded once (2^-24).  A factor 1 and an addend 0 add nothing.
The oracle's 64-bit sine of a reduced angle is good to 1e-15."""
import math
from fractions import Fraction

import pytest
import torch

from paged_kv_cache_456_b200 import ops

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_456_b200 import build
    build.build()
    ops.library()


def exact(pos, freq):
    theta = Fraction(pos) * Fraction(freq)
    theta -= round(theta / TWO_PI) * TWO_PI
    return math.cos(theta), math.sin(theta)


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32), (80, 80)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("far", [1, 4096, 1 << 20, 1 << 31, 1 << 40, (1 << 53) - 1])
def test_cosine_and_sine_at_any_distance(D, rot, adjacent, far):
    T, half = 24, rot // 2
    g = torch.Generator().manual_seed(far % 1000003 + D)
    pos = torch.cat([torch.tensor([0, 1, -1, far, -far, far - 1]),
                     torch.randint(-far, far + 1, (T - 6,), generator=g)])
    freq = (10000.0 ** (-torch.arange(half).double() / half)).float()
    freq[-1] = math.pi       # (turns an odd position by almost half a turn: a sine of next to nothing)
    freq[-2] = math.pi / 2
    freq[-3] = 37.5
    x = torch.zeros(T, 1, D)
    x[..., 0:rot:2 if adjacent else 1][..., :half] = 1.0
    out = ops.rope_append(torch.empty(T, 1, D, device="cuda"), x.cuda(), None, None, None, None, None, pos.cuda(), freq.cuda(),
                          adjacent=adjacent).cpu().double()[:, 0]
    cos, sin = (out[:, 0:rot:2], out[:, 1:rot:2]) if adjacent else (out[:, :half], out[:, half:rot])
    want = torch.tensor([[exact(p, f) for f in freq.tolist()] for p in pos.tolist()], dtype=torch.float64)
    for got, ref in ((cos, want[..., 0]), (sin, want[..., 1])):
        err, bound = (got - ref).abs(), (2.0 ** -23 + 2.0 ** -24) * ref.abs() + 2.0 ** -45
        assert (err <= bound).all(), f"worst error / bound {(err / bound).max():.3f}, error {err.max():.2e}"


def test_the_farthest_positions_there_are():
    """Past 2^53 a position counts as the double nearest to it: the angle is that double's."""
    far = [(1 << 63) - 1, -(1 << 63), (1 << 53) + 1, (1 << 60) + 12345, -(1 << 62) - 1]
    freq = [1.0, 0.5, 0.001, 3.0e-5, 2.0 ** -40, 0.0, 7.0, 1.0e-20]
    pos = torch.tensor(far)
    x = torch.zeros(len(far), 1, 16)
    x[..., :8] = 1.0
    out = ops.rope_append(torch.empty(len(far), 1, 16, device="cuda"), x.cuda(), None, None, None, None, None, pos.cuda(),
                          torch.tensor(freq, device="cuda")).cpu().double()[:, 0]
    want = torch.tensor([[exact(float(p), f) for f in torch.tensor(freq).tolist()] for p in far], dtype=torch.float64)
    # two doubles hold a fraction of a turn of 2^63 radians to about 2^63 2^-104
    for got, ref in ((out[:, :8], want[..., 0]), (out[:, 8:], want[..., 1])):
        assert ((got - ref).abs() <= (2.0 ** -23 + 2.0 ** -24) * ref.abs() + 2.0 ** -39).all()
