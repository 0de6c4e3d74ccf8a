"""pa_rope_append in the shapes that large calls take: several rounds of rows a warp, more data than the L2 holds, and
several tokens a CTA for heads that do not divide a warp.  Definition and tolerance as in test_gpu_rope."""
import pytest
import torch

from paged_kv_cache_456_b200 import ops

from tests.test_gpu_rope import assert_turned, bits, call, check, inputs, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_456_b200 import build
    build.build()
    ops.library()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes", [
    (2048, 64, 8, 128, 128, 1), (2048, 61, 5, 128, 96, 1),      # 20 and 18 rounds of four rows, the last in part
    (2500, 12, 4, 128, 128, 3), (2501, 7, 3, 64, 32, 1),        # more tokens than have a place at once
    (900, 33, 2, 256, 64, 2), (2400, 9, 1, 512, 512, 1)])
def test_several_rounds_of_rows(dtype, adjacent, T, Hq, Hkv, D, rot, axes):
    check(inputs(T, Hq, Hkv, D, rot, dtype=dtype, axes=axes, padding=T // 9), adjacent)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype,T", [("bf16", 6001), ("f32", 3001)])
def test_more_than_the_l2_holds(dtype, T, adjacent):
    """147 MB read and written: the streaming loads and stores."""
    x = inputs(T, 32, 8, 128, 128, dtype=dtype, axes=3, padding=50)
    check(x, adjacent)
    apart = torch.empty_like(x["q"])
    assert call(x, apart, adjacent=adjacent) == 0
    assert call(x, x["q"], adjacent=adjacent) == 0      # and in place
    assert torch.equal(bits(x["q"]), bits(apart))


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T", [2048, 2600])
def test_in_place_over_several_rounds(T, adjacent):
    x = inputs(T, 40, 4, 128, 64)
    apart = torch.empty_like(x["q"])
    assert call(x, apart, adjacent=adjacent) == 0
    assert call(x, x["q"], adjacent=adjacent) == 0
    assert torch.equal(bits(x["q"]), bits(apart))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (3001, 12, 4, 80, 48), (9003, 4, 1, 96, 96), (9001, 3, 2, 72, 16), (4000, 1, 1, 24, 16), (20011, 2, 1, 80, 80)])
def test_several_tokens_a_cta(dtype, adjacent, T, Hq, Hkv, D, rot):
    """Heads whose units do not divide a warp, with tokens enough for several a CTA, the last CTA in part."""
    check(inputs(T, Hq, Hkv, D, rot, dtype=dtype, padding=T // 11), adjacent)


def test_several_tokens_a_cta_with_bad_slots():
    x = inputs(3001, 12, 4, 80, 80)
    want, slack = turned(x["q"], x["positions"], x["inv_freq"], None, False, 1.0)
    x["slots"][::5] = x["k_cache"].shape[0] * 16
    k0 = x["k_cache"].clone()
    q_out = torch.empty_like(x["q"])
    assert call(x, q_out) == ops.ERRBIT_SLOT
    assert_turned(q_out, want, slack)
    changed = (bits(x["k_cache"]) != bits(k0)).any(dim=3).any(dim=1).sum().item()
    assert 0 < changed <= 3001 - len(range(0, 3001, 5))
