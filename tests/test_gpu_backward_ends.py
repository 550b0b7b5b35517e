"""The gradient's reverse scan over rings of stages that are used not at all, once, as often
as there are stages, and more often, in calls that follow one another without a pause."""
import pytest
import torch

from test_gpu_backward import TOL, check, falcon, ref_bwd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rule", ["falcon1", "falcon1a"])
@pytest.mark.parametrize("heads", [3, 200])
def test_rows_of_one_to_nine_chunks(falcon, rule, heads):  # noqa: F811
    fn = falcon.falcon1_bwd_chunked if rule == "falcon1" else falcon.falcon1a_bwd_chunked
    for chunks in range(1, 10):
        T = 64 * chunks - 7
        g = torch.Generator(device="cuda").manual_seed(T)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        x = {n: r(1, heads, T, 64).bfloat16() for n in ("q", "k", "v")}
        x["beta"] = torch.rand(1, heads, T, generator=g, device="cuda")
        x["lambda"] = 0.1 * torch.rand(1, heads, T, generator=g, device="cuda")
        dO = r(1, heads, T, 64).bfloat16()
        runs = [fn(x["q"], x["k"], x["v"], x["beta"], x["lambda"], dO) for _ in range(4)]
        assert falcon.falcon_sync_check() == 0
        for again in runs[1:]:
            assert torch.equal(again["dq"], runs[0]["dq"])
            assert torch.equal(again["dS0"], runs[0]["dS0"])
            # sums whose order varies: the last bits, and now and then a rounding to bf16
            for n in ("dk", "dv", "dbeta", "dlambda"):
                a, b = again[n].double(), runs[0][n].double()
                assert float((a - b).norm() / b.norm()) < 1e-5, n
        few = {n: t[:, :3].contiguous() for n, t in x.items()}
        ref = ref_bwd(rule, few, dict(dO=dO[:, :3].contiguous()), "l2")
        got = {n: t[:, :3].float().cpu().numpy() for n, t in runs[0].items() if t is not None}
        check(got, ref, TOL[torch.bfloat16], ("dq", "dk", "dv", "dbeta", "dlambda"))
