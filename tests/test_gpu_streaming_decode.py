"""The example's decode loop on the GPU: append, attend, quantize and evict_step together."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decode_harness import attend64  # noqa: E402

pytestmark = pytest.mark.gpu


def _decoder(**kw):
    from streaming_decode import StreamingDecoder
    return StreamingDecoder(**kw)


def _tokens(n, width, seed, seqs=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(seqs, n, width, generator=g, device="cuda").bfloat16()


def test_chunks_and_single_tokens_give_one_forward_pass():
    # 96 tokens at once against chunks of 33, 1, 1, 40 and 21 of the same tokens: the only
    # difference is the order of sums and one rounding to bf16 per stage (2^-8 of values of
    # order 1, over 2 layers of 5 stages)
    whole = _decoder(budget=128, slack=32, chunk=128)
    parts = _decoder(budget=128, slack=32, chunk=128)
    x = _tokens(96, 2 * 4 * 128, 3)
    a = whole.forward(x)
    b = torch.cat([parts.forward(y) for y in x.split([33, 1, 1, 40, 21], dim=1)], dim=1)
    whole.check()
    parts.check()
    assert torch.equal(whole.cache.lens, parts.cache.lens)
    assert (a.float() - b.float()).norm() <= 10 * 2.0 ** -8 * a.float().norm()


@pytest.mark.parametrize("image", [False, True])
def test_loop_stays_within_its_budget_and_reads_what_it_holds(image):
    m = _decoder(budget=128, slack=32, chunk=64, image=image)
    width = 2 * 4 * 128
    for i in range(6):
        m.forward(_tokens(64, width, i))
    for i in range(80):
        m.forward(_tokens(1, width, 100 + i))
    m.check()
    assert m.evictions >= 3 and m.held <= 128 + 32 + 64
    assert torch.all(m.cache.lens == m.held)
    T = m.held
    pos = m.cache.pos[..., :T]
    assert torch.all(pos[..., 1:] > pos[..., :-1])                   # survivors in their order
    assert torch.all(pos[..., -1] == m.position - 1)
    if image:
        assert torch.all(m.image.rows == T // 32 * 32)
    # the last query of layer 0 over the rows that its cache holds now
    from streaming_kv_cache_step_gb300 import nexus
    q = m.queries[0, :, :, -1].contiguous()
    out = torch.empty_like(q)
    nexus.attend(m.cache, 0, q, out, m.attend_ws, m.status, max_tokens=1, image=m.image)
    m.check()
    for s in range(2):
        for h in range(2):
            k, v = m.cache.k[0, s, h, :T].double().cpu(), m.cache.v[0, s, h, :T].double().cpu()
            r = T // 32 * 32 if image else 0
            if r:
                for t, c, sc in ((k, m.image.k, m.image.k_scale), (v, m.image.v, m.image.v_scale)):
                    t[:r] = c[0, s, h].float()[:r].double().cpu() * \
                        sc[0, s, h, :r // 32].double().cpu().repeat_interleave(32)[:, None]
            rows = q[s, 4 * h:4 * h + 4].cpu()
            ref, _, A, big = attend64(rows, k, v, [T] * 4, 128 ** -0.5)
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * 2.0 ** -24 * 136 * 128 ** -0.5 * big)[:, None] * A
            assert torch.all((out[s, 4 * h:4 * h + 4].double().cpu() - ref).abs() <= tol)


def test_example_runs():
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for extra in ([], ["--image"]):
        p = subprocess.run([sys.executable, os.path.join(root, "examples", "streaming_decode.py"),
                            "--layers", "2", "--prompt", "700", "--tokens", "70", "--budget", "256",
                            "--slack", "32", "--chunk", "256", *extra], capture_output=True,
                           text=True, timeout=300)
        assert p.returncode == 0, p.stderr
        assert "evictions" in p.stdout
