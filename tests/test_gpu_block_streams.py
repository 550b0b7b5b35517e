"""Calls on a given stream while the current one is busy with memory that it has already
given back to the allocator."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_results_of_a_call_on_another_stream_are_not_in_memory_still_in_use():
    import delta_rule_attention_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    B, T, D, N = 2, 600, 256, 16
    d = dict(u=r(B, T, D), delta=r(B, T, D), A=-torch.exp(r(D, N)), Bm=r(B, T, 1, N),
             Cm=r(B, T, 1, N), D=r(D), z=r(B, T, D))
    dy, w = r(B, T, D), r(D, 4)
    grads = m.falcon_selective_scan_bwd(**d, dy=dy)
    conv = m.falcon_short_conv_bwd(d["u"], w, dy)
    y, h = m.falcon_selective_scan_fwd(**d)
    sizes = sorted({t.numel() for out in (grads, conv) for t in out.values() if t is not None}
                   | {y.numel(), h.numel(), 1 << 20, 5 << 20})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        # what the current stream will write to, and has given back
        held = [torch.empty(n, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in held:
            t.fill_(float("nan"))
        del held, t
        got = m.falcon_selective_scan_bwd(**d, dy=dy, stream=side)
        cg = m.falcon_short_conv_bwd(d["u"], w, dy, stream=side)
        y1, h1 = m.falcon_selective_scan_fwd(**d, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], grads[k]) for k in grads if grads[k] is not None)
        assert all(torch.equal(cg[k], conv[k]) for k in conv)
        assert torch.equal(y, y1) and torch.equal(h, h1)


def test_results_may_be_dropped_while_the_current_stream_reads_them():
    import delta_rule_attention_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.randn(2, 700, 512, generator=g, device="cuda"), torch.ones(512, 4, device="cuda")
    want, other = m.falcon_short_conv_fwd(x, w)[0].clone(), 2 * w
    torch.cuda.synchronize()
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    y, tail = m.falcon_short_conv_fwd(x, w, stream=side)
    here.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept = y.clone()  # queued behind the wait
    del y, tail
    for _ in range(4):  # would take y's memory and write to it at once
        m.falcon_short_conv_fwd(x, other, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_calls_on_a_given_stream_inside_a_graph():
    import delta_rule_attention_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    B, T, D, N = 2, 90, 64, 16
    d = dict(u=r(B, T, D), delta=r(B, T, D), A=-torch.exp(r(D, N)), Bm=r(B, T, 1, N),
             Cm=r(B, T, 1, N), D=r(D), z=r(B, T, D))
    dy, w = r(B, T, D), r(D, 4)

    def both(**on):
        x, _ = m.falcon_short_conv_fwd(d["u"], w, **on)
        y, h = m.falcon_selective_scan_fwd(**{**d, "u": x}, **on)
        grads = m.falcon_selective_scan_bwd(**{**d, "u": x}, dy=dy, **on)
        norm = m.falcon_clip_grad_norm([grads["dA"], grads["dB"]], 1.0, **on)
        return y, h, grads["du"], grads["dA"], grads["dB"], norm

    want = [t.clone() for t in both()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = both(stream=side)
        here.wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
