"""Sparse decoding of a batch of sessions on paged cache rows.

    python examples/sparse_decode.py [--sessions 4] [--prompt 5000] [--steps 8] [--k 2048] [--block 1]

Every session's rows live in the blocks of a session pool, its index keys next
to them.  A prompt is appended in one call; then, per step and for all
sessions at once:

    append_tokens     the new token's latent, position part and index key become a cache row and key
    index_scores      the cheap score of every cached position (or of every block of positions)
    select_topk_batch the best k of them
    attend            attention over the rows of the selected positions (or blocks)

The steps run as one captured CUDA graph.  The model around them is random:
this shows the calls, their shapes and their order.  Prints what a step takes,
and how near attention over the selection comes to attention over everything.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gather_radix_top_gb300 import build, kvo  # noqa: E402

HEADS, INDEX_HEADS, SCALE = 64, 32, 192 ** -0.5
INV_FREQ = 10_000.0 ** (-torch.arange(0, kvo.ROPE_VALUES, 2, dtype=torch.float64) / kvo.ROPE_VALUES)


def decode(sessions: int = 4, prompt: int = 5_000, steps: int = 8, k: int = 2_048, block: int = 1, seed: int = 0) -> dict:
    """Runs `steps` decode steps; returns the last step's selection, output and the checks' figures."""
    build.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    total = prompt + steps
    blocks = -(-total // 16)
    with kvo.Context(layers=1, history_cap=64, hot_rows=64) as ctx, \
            kvo.Pool(layers=1, pool_blocks=sessions * blocks, block_tokens=16, tier_blocks=0) as pool:
        for s in range(sessions):
            assert pool.alloc(s, total) == kvo.KVO_OK
        table = torch.tensor([kvo.kvo_pool_block_table(pool.handle, s, 0) for s in range(sessions)],
                             dtype=torch.int32, device="cuda")
        rows = sessions * blocks * 16
        keys = torch.zeros(rows, kvo.KEY_VALUES, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        cache = kvo.Cache(rows=pool, keys=keys, key_scales=torch.zeros(rows, device="cuda"), table=table)

        # the prompt: all sessions' tokens in one call
        kv, key = rand(sessions * prompt, 576).bfloat16(), rand(sessions * prompt, kvo.KEY_VALUES).bfloat16()
        seq = torch.arange(sessions, dtype=torch.int32, device="cuda").repeat_interleave(prompt)
        pos = torch.arange(prompt, dtype=torch.int32, device="cuda").repeat(sessions)
        ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], pos, INV_FREQ, seq=seq, key=key)

        # one step's buffers; a model would write the inputs, here they are drawn between the steps
        units = min(k, total) if block == 1 else min(k // block, -(-total // block))
        st = dict(kv=rand(sessions, 576).bfloat16(), key=rand(sessions, kvo.KEY_VALUES).bfloat16(),
                  qi=rand(sessions, INDEX_HEADS, kvo.KEY_VALUES).to(torch.float8_e4m3fn),
                  w=rand(sessions, INDEX_HEADS).abs(), q=rand(sessions, HEADS, 576).bfloat16(),
                  pos=torch.full((sessions,), prompt, dtype=torch.int32, device="cuda"),
                  lens=torch.full((sessions,), prompt + 1, dtype=torch.int32, device="cuda"),
                  scores=torch.empty(sessions, -(-total // block), device="cuda"),
                  idx=torch.empty(sessions, units, dtype=torch.int32, device="cuda"),
                  out=torch.empty(sessions, HEADS, 512, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(sessions, HEADS, device="cuda"))
        need = kvo.kvo_attend_work_bytes(sessions, HEADS, units * block)
        work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

        def step():
            ctx.append_tokens(cache, st["kv"][:, :512], st["kv"][:, 512:], st["pos"], INV_FREQ, key=st["key"])
            ctx.index_scores(cache, st["qi"], st["w"], st["lens"], total, block=block, out=st["scores"])
            ctx.select_topk_batch(st["scores"], units, idx=st["idx"])
            ctx.attend(cache, st["q"], st["lens"], SCALE, sel=st["idx"], sel_block=block, out=st["out"], lse=st["lse"],
                       work=work)

        step()                                    # before the capture: loads the kernels
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        spent = 0.0
        for i in range(steps):
            st["kv"].copy_(rand(sessions, 576))
            st["key"].copy_(rand(sessions, kvo.KEY_VALUES))
            st["qi"].copy_(rand(sessions, INDEX_HEADS, kvo.KEY_VALUES).to(torch.float8_e4m3fn))
            st["q"].copy_(rand(sessions, HEADS, 576))
            st["pos"].fill_(prompt + i)
            st["lens"].fill_(prompt + i + 1)
            begin.record()
            graph.replay()
            end.record()
            end.synchronize()
            spent += begin.elapsed_time(end)
        # how much of the whole softmax the selection holds
        _, lse = ctx.attend(cache, st["q"], st["lens"], SCALE, rows=total)
        assert ctx.sync() == kvo.KVO_OK
        return dict(us_per_step=1e3 * spent / max(steps, 1), idx=st["idx"].clone(), out=st["out"].clone(),
                    share=float(torch.exp(st["lse"] - lse).mean()), q=st["q"].clone(), lens=st["lens"].clone(),
                    lse=st["lse"].clone(), all_lse=lse.clone())


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("sessions", 4), ("prompt", 5_000), ("steps", 8), ("k", 2_048), ("block", 1)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    r = decode(a.sessions, a.prompt, a.steps, a.k, a.block)
    print(f"{a.sessions} sessions, {a.prompt + a.steps} positions: {r['us_per_step']:.1f} us a step "
          f"(append, scores, top-k, attention); the selection holds {100 * r['share']:.1f} % of the softmax")


if __name__ == "__main__":
    main()
