"""The holder classes over several calls: what they report and answer does not depend on the way a
forward was started."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests.test_gpu_operators import CU, few_case, same_bits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


def test_last_error_is_of_the_forward_that_ran():
    """MegaMoE.last_error counts the routes that the newest forward on the GPU dropped: capturing
    forward_few runs nothing, and replaying it does, whatever was called from Python last."""
    M, K, E, top_k, I = 4, 256, 8, 2, 128
    w, inp, dev, d, _, _ = few_case(M, K, E, top_k, I, seed=3)
    moe = MM.MegaMoE(M, K, E, top_k, I)
    moe.load_weights(dev["w1"], dev["scale1"], dev["w2"], dev["scale2"])
    one, three = dev["expert_idx"].clone(), dev["expert_idx"].clone()
    one[0, 0] = -1
    three[1:, 1] = E
    few_out = torch.empty((M, K), dtype=torch.bfloat16, **CU)
    want_one = moe.forward(dev["x"], one, dev["probs"])
    assert moe.last_error() == 1
    want_three = moe.forward_few(dev["x"], three, dev["probs"])
    assert moe.last_error() == 3

    moe.forward(dev["x"], one, dev["probs"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward_few(dev["x"], three, dev["probs"], out=few_out)
    assert moe.last_error() == 1, "the capture has run nothing"
    for _ in range(3):
        few_out.fill_(float("nan"))
        graph.replay()
        assert moe.last_error() == 3 and same_bits(few_out, want_three)
        # the two forms in turn find nothing of each other's in the workspace
        assert same_bits(moe.forward(dev["x"], one, dev["probs"]), want_one)
        assert moe.last_error() == 1
    whole = torch.cuda.CUDAGraph()
    out = torch.empty_like(few_out)
    with torch.cuda.graph(whole):
        moe.forward(dev["x"], one, dev["probs"], out=out)
    moe.forward_few(dev["x"], three, dev["probs"])
    for _ in range(3):
        whole.replay()
        assert moe.last_error() == 1 and same_bits(out, want_one)
        assert same_bits(moe.forward_few(dev["x"], three, dev["probs"]), want_three)
        assert moe.last_error() == 3


def test_forward_before_the_weights():
    """Without weights the int8 forms are refused with the library's error and the MXFP4 layer
    answers NaN; weights that are refused leave the ones before them whole."""
    M, K, E, top_k, I = 4, 256, 8, 2, 128
    x = torch.ones((M, K), dtype=torch.float16, **CU)
    ids = torch.arange(M * top_k, dtype=torch.int32, **CU).view(M, top_k)
    probs = torch.full((M, top_k), 0.5, **CU)
    moe = MM.MegaMoE(M, K, E, top_k, I)
    for form in (moe.forward, moe.forward_few):
        with pytest.raises(MM.MegaMoEError) as err:
            form(x, ids, probs)
        assert err.value.status == 1

    # the allocator hands out memory that held finite values before
    for shape in ((E, 2 * I, K // 2), (E, 2 * I, K // 32), (E, K, I // 2), (E, K, I // 32)):
        torch.full(shape, 120, dtype=torch.uint8, **CU)
    mx = MM.MegaMoEMXFP4(M, K, E, top_k, I)
    assert torch.isnan(mx.forward(x, ids, probs)).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, w2 = torch.randn((E, 2 * I, K), generator=g, **CU) / 16, torch.randn((E, K, I), generator=g, **CU) / 11
    mx.load_weights(w1, w2)
    want = mx.forward(x, ids, probs)
    assert torch.isfinite(want).all() and (want != 0).any()
    for bad, error in ((w2[:, :-1], ValueError), (w2.cpu(), ValueError), (w2.double(), TypeError)):
        with pytest.raises(error):
            mx.load_weights(w1 * 2, bad)
        assert same_bits(mx.forward(x, ids, probs), want)
    wide = torch.zeros((E, K, 2 * I), **CU)
    wide[..., ::2] = w2
    mx.load_weights(w1, wide[..., ::2])    # of any strides
    assert same_bits(mx.forward(x, ids, probs), want)
