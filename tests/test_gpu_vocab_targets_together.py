"""GPU tests of the cross entropy's gradients with dW's exact target elements (tokens sorted by target and summed beside the
product) in captured graphs and on two streams: every result equals the eager call's bit for bit."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
# sums per token, by counting and by radix; per row of one of two pieces
SIZES = [(8192, 16384, 128), (20000, 4096, 256), (65536, 16384, 32)]


def state(device, tokens, vocab, width, key):
    gen = torch.Generator(device=device).manual_seed(tokens + key)
    u = torch.rand(tokens, generator=gen, device=device, dtype=torch.float64)
    y = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1)
    y[::5] = -100
    return {"H": torch.randn(tokens, width, generator=gen, device=device).to(BF16),
            "W": (torch.randn(vocab, width, generator=gen, device=device) * width ** -0.5).to(BF16), "y": y,
            "g": torch.rand(tokens, generator=gen, device=device)}


def run(dion, s, out, stream=None):
    dion.linear_cross_entropy_(s["H"], s["W"], s["y"], loss=out["loss"], lse=out["lse"], workspace=out["w1"], stream=stream)
    dion.linear_cross_entropy_grad_(s["H"], s["W"], s["y"], out["lse"], s["g"], out["dH"], out["dW"], workspace=out["w2"],
                                    stream=stream)


def outputs(dion, s):
    (vocab, width), tokens, device = s["W"].shape, s["y"].numel(), s["W"].device
    return {"loss": torch.empty(tokens, device=device), "lse": torch.empty(tokens, device=device),
            "dH": torch.empty_like(s["H"]), "dW": torch.empty_like(s["W"]),
            "w1": dion.linear_cross_entropy_workspace_for(tokens, vocab, width, device, BF16).fill_(255),
            "w2": dion.linear_cross_entropy_workspace_for(tokens, vocab, width, device, BF16, for_grad=True).fill_(255)}


RESULTS = ("loss", "lse", "dH", "dW")


@pytest.mark.parametrize("tokens,vocab,width", SIZES)
def test_replays_equal_eager_calls(cuda, tokens, vocab, width):
    import rank_orthonormalized_optimizer_amd as dion
    states = [state(cuda, tokens, vocab, width, k) for k in range(2)]
    want = []
    for s in states:
        out = outputs(dion, s)
        run(dion, s, out)
        want.append({k: out[k] for k in RESULTS})
    held = {k: v.clone() for k, v in states[0].items()}
    out = outputs(dion, held)
    torch.cuda.synchronize()
    print(f"[targets] graph of {tokens} x {vocab} x {width}", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(dion, held, out)
    for k in (1, 0, 1):
        for name in held:
            held[name].copy_(states[k][name])
        out["w1"].fill_(255)
        out["w2"].fill_(255)
        graph.replay()
        eager = outputs(dion, states[1 - k])
        run(dion, states[1 - k], eager)
        torch.cuda.synchronize()
        for name in RESULTS:
            assert torch.equal(out[name], want[k][name]), f"replay of {k}: {name}"
            assert torch.equal(eager[name], want[1 - k][name]), f"beside it: {name}"


def test_two_streams_at_once(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    states = [state(cuda, *SIZES[0], k) for k in range(2)]
    want = [outputs(dion, s) for s in states]
    for s, out in zip(states, want):
        run(dion, s, out)
    streams = [torch.cuda.Stream() for _ in states]
    got = [outputs(dion, s) for s in states]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, out, stream in zip(states, got, streams):
            run(dion, s, out, stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in RESULTS)


@pytest.mark.parametrize("tokens,vocab,width", SIZES)
def test_int32_targets_and_an_ignored_id_of_the_vocabulary(cuda, tokens, vocab, width):
    """int32 and int64 targets give the same bits; an ignored id that is a row of W leaves nothing in that row but the
    probabilities of the others, and a target outside the vocabulary makes dW NaN."""
    import rank_orthonormalized_optimizer_amd as dion
    s = state(cuda, tokens, vocab, width, 5)
    y = s["y"].clamp(min=0)          # the ignored ones become targets of id 0, the most frequent one
    one = torch.full((1,), 1.0 / tokens, device=cuda)

    def grads(targets, ignore):
        _, lse = dion.linear_cross_entropy_(s["H"], s["W"], targets, ignore_index=ignore)
        dH, dW = torch.empty_like(s["H"]), torch.empty_like(s["W"])
        dion.linear_cross_entropy_grad_(s["H"], s["W"], targets, lse, one, dH, dW, ignore_index=ignore)
        return dH, dW

    dH, dW = grads(y, 0)
    for a, b in zip((dH, dW), grads(y.to(torch.int32), 0)):
        assert torch.equal(a, b)
    for a, b in zip((dH, dW), grads(torch.where(y == 0, -100, y), -100)):
        assert torch.equal(a, b)
    assert not dH[y == 0].any() and torch.isfinite(dW.float()).all()
    y[3] = vocab
    dH, dW = grads(y, 0)
    assert torch.isnan(dW).all() and torch.isnan(dH[3]).all() and torch.isfinite(dH[4:].float()).all()
