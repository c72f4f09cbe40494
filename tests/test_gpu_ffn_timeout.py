"""Bounded waits that run out: the kernels end by themselves, say so in the
handle's status, leave no plausible sums where partial ones are joined, and
the handle works on."""
import pytest
import torch

from tests import _ffn_reference as R
from tests._harness import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _bf16(T, d, F, ops):
    g = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()
    W = {"gate": rnd(F, d, std=d ** -0.5), "up": rnd(F, d, std=d ** -0.5), "down": rnd(d, F, std=F ** -0.5)}
    return ops.GatedFFN(W, max_tokens=T), (rnd(T, d),)


def _mx(T, d, F, ops):
    g = torch.Generator(device="cuda").manual_seed(T)
    W = {}
    for n, o, i in (("gate", F, d), ("up", F, d), ("down", d, F)):
        W[n], W[n + "_s"] = R.mx_random((o, i), i ** -0.5, g, "cuda")
    return ops.GatedFFN(W, max_tokens=T), R.mx_random((T, d), 1.0, g, "cuda")


# streamed weights (K a multiple of 64, and not; one CTA and eight of a cluster), K split over pairs, whole pair tiles
@pytest.mark.parametrize("make,T,d,F,joined", [
    (_bf16, 3, 64, 64, True), (_bf16, 3, 1024, 256, True), (_bf16, 20, 1096, 136, True), (_bf16, 72, 2048, 256, True),
    (_bf16, 300, 256, 256, True), (_bf16, 130, 1024, 256, True), (_bf16, 1000, 512, 1024, False),
    (_mx, 5, 128, 64, True), (_mx, 5, 2048, 192, True), (_mx, 40, 1056, 96, True), (_mx, 300, 256, 192, False)])
def test_wait_that_runs_out(ops, make, T, d, F, joined):
    layer, x = make(T, d, F, ops)
    call = layer.lmoe_ffn_forward_mx if layer.mx else layer.lmoe_ffn_forward
    want = call(*x)
    layer.lmoe_ffn_sync_status()
    y = layer.lmoe_ffn_selftest_timeout(*x)
    with pytest.raises(ops.LmoeError) as e:
        layer.lmoe_ffn_sync_status()
    assert e.value.status == ops.LMOE_ERR_TIMEOUT
    if joined:
        assert bool(torch.isnan(y).all())
    layer.lmoe_ffn_sync_status()                # the flag is cleared
    assert torch.equal(call(*x), want)
    layer.lmoe_ffn_sync_status()
    layer.close()


# rows of one warp and of many, several groups of warps, one and five vectors per thread
@pytest.mark.parametrize("T,d", [(40000, 256), (4000, 7168), (2000, 8192), (600, 16384)])
def test_norm_rows_that_never_are_complete(ops, T, d):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    want = ops.lmoe_add_rms_norm(x, w, 1e-6)[0]
    dwant = ops.lmoe_add_rms_norm_backward(x, x, w, 1e-6)
    y, _ = ops.lmoe_add_rms_norm_selftest_timeout(x, w)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y).all())
    dx, dw = ops.lmoe_add_rms_norm_selftest_timeout(x, w, backward=True)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dx).all()) and bool(torch.isnan(dw).all())
    assert torch.equal(ops.lmoe_add_rms_norm(x, w, 1e-6)[0], want)
    got = ops.lmoe_add_rms_norm_backward(x, x, w, 1e-6)
    assert torch.equal(got[0], dwant[0]) and torch.equal(got[1], dwant[1])
