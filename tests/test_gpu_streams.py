"""The bf16 entry points on a stream of the caller's, with outputs and workspaces of their own: neither what they
fill nor what they allocate is left to the current stream, and work that is queued there keeps its memory."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def uocr(cuda_device):
    import block_sparse_long_uocr_b200 as m
    return m


def test_calls_on_another_stream_beside_a_busy_current_one(uocr, cuda_device):
    total, n = 4000, 40
    c = workloads.make_case([total, 700], shuffle=True, seed=3, device=cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    rnd = lambda *shape: torch.randn(shape, generator=g, device=cuda_device).to(torch.bfloat16)  # noqa: E731
    q, iq = rnd(n, *c.q.shape[1:]), rnd(n, 128)
    pos = torch.arange(total - n, total, dtype=torch.int32, device=cuda_device)
    bt, sl, kv = c.block_table, c.seq_lens, (c.k_pool, c.v_pool)
    summary = rnd(c.idx_k_pool.shape[0], 128)
    scores = uocr.index_score(c.idx_q, c.idx_k_pool, bt, sl)
    sel = uocr.block_topk(scores, sl)
    many = uocr.sparse_prefill(q, *kv, iq, c.idx_k_pool, bt, sl, 0, pos)[1]
    mask = torch.full((2, -(-bt.shape[1] // 32)), -1, dtype=torch.int32, device=cuda_device)
    calls = {
        "index_score": lambda s: uocr.index_score(c.idx_q, c.idx_k_pool, bt, sl, stream=s),
        "block_topk": lambda s: uocr.block_topk(scores, sl, stream=s),
        "block_topk_masked": lambda s: uocr.block_topk_masked(scores, sl, mask, stream=s),
        "sparse_attn": lambda s: uocr.sparse_attn(c.q, *kv, bt, sl, sel, stream=s),
        "sparse_decode": lambda s: uocr.sparse_decode(c.q, *kv, c.idx_q, c.idx_k_pool, bt, sl, stream=s),
        "prefill_index_score": lambda s: uocr.prefill_index_score(iq, c.idx_k_pool, bt, sl, 0, pos, stream=s),
        "sparse_prefill": lambda s: uocr.sparse_prefill(q, *kv, iq, c.idx_k_pool, bt, sl, 0, pos, stream=s),
        "sparse_attn_seq": lambda s: uocr.sparse_attn_seq(q, *kv, bt, sl, 0, pos, many, stream=s),
        "summary_score": lambda s: uocr.summary_score(c.idx_q, summary, bt, sl, stream=s),
        "block_summary_mean": lambda s: uocr.block_summary_mean(c.idx_k_pool, stream=s),
        "sparse_decode_summary": lambda s: uocr.sparse_decode_summary(c.q, *kv, c.idx_q, summary, bt, sl, stream=s),
        "dense_decode": lambda s: uocr.dense_decode(c.q, *kv, bt, sl, stream=s),
    }
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in calls.items():
        as_tuple = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
        want = [x.clone() for x in as_tuple(call(None))]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        temps = [torch.full((x.numel() * x.element_size(),), 0x5A, dtype=torch.uint8, device=cuda_device) for x in want]
        keep = [torch.zeros_like(t) for t in temps]
        torch.cuda.synchronize()
        torch.cuda._sleep(80_000_000)
        for a, b in zip(keep, temps):
            a.copy_(b)
        del temps, a, b
        got = as_tuple(call(side))
        side.synchronize()
        assert not torch.cuda.current_stream().query(), "the current stream was done before the call on the other"
        with torch.cuda.stream(side):
            same = all(bool(torch.equal(x, y)) for x, y in zip(got, want))   # before the current stream goes on
        torch.cuda.synchronize()
        assert same and all((x == 0x5A).all() for x in keep), name
        torch.cuda._sleep(20_000_000)
        later = [x.clone() for x in got]
        del got
        other = as_tuple(call(side))
        with torch.cuda.stream(side):
            for x in other:
                x.zero_()
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(later, want)), name
