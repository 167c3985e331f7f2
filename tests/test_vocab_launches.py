"""The grids of the vocabulary operators' launches: every size that is accepted fits HIP's limits (on the CPU, under the
sanitizers), and passes that stride over their items reach all of them (on the GPU)."""
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VOCAB = os.path.join(ROOT, "rank_orthonormalized_optimizer_amd", "csrc", "vocab")


def test_every_grid_fits(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "vocab_launches")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
           os.path.join(ROOT, "include"), "-I", VOCAB, os.path.join(ROOT, "tests", "host_san", "vocab_launches.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=240)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    out = run.stdout + run.stderr
    assert run.returncode == 0 and "every grid fits" in out and "runtime error" not in out, out[-3000:]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_more_outputs_than_a_grid_takes(cuda, dt):
    """dH of 65792 x 1040 from two pieces of the vocabulary: its last pass has 68.4e6 outputs, four for each of 65536 x 256
    threads and some for a second round.  A token's dH does not depend on the others: the first, the last and those at the
    border of the rounds, alone in a call of few tokens, are the same up to both calls' bounds."""
    import rank_orthonormalized_optimizer_amd as dion
    from tests.vocab_reference import Head
    tokens, vocab, width = 65792, 8500, 1040
    gen = torch.Generator(device=cuda).manual_seed(2)
    W = (torch.randn(vocab, width, generator=gen, device=cuda) / 32).to(dt)
    H = torch.randn(tokens, width, generator=gen, device=cuda).to(dt)
    y = torch.randint(0, vocab, (tokens,), generator=gen, device=cuda)
    _, lse = dion.linear_cross_entropy_(H, W, y)
    dH = torch.full_like(H, float("nan"))
    one = torch.ones(1, device=cuda)
    dion.linear_cross_entropy_grad_(H, W, y, lse, one, dH)
    border = 65536 * 256 * 4 // width
    some = torch.cat([torch.arange(a, a + 50, device=cuda) for a in (0, border - 25, tokens - 50)])
    want = Head(H[some], W, y[some], grad=one)
    off = (dH[some].double() - want.dH).abs()
    assert bool((off <= want.dH_bound).all()), float((off / want.dH_bound).max())
    assert torch.isfinite(dH.float().sum())
