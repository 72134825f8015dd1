"""QuantizedPagedDecoder over an 8-bit cache, its own work on the CPU: the library's calls replaced by records."""
import pytest
import torch

import query_aware_sparse_kv_gb300 as qskv
from query_aware_sparse_kv_gb300 import engine
from test_kvq_engine import _held, _state, _tokens, calls as calls4  # noqa: F401

HQ, HKV, D = 4, 2, 64


@pytest.fixture
def calls(calls4, monkeypatch):
    """The calls that a decoder of 8 bits makes; the prefill refuses token strides as the library does."""
    def record(name, fn=None):
        def call(*args, **kw):
            calls4.append((name, args, kw))
            return fn(*args, **kw) if fn else None

        monkeypatch.setattr(engine.B, name, call)

    def prefill(q, *args, **kw):
        if len(q) > 1 and q.stride(0) < q.shape[1] * q.shape[2]:
            raise qskv.QskvError(1, "q_stride must be at least num_q_heads * head_dim and a multiple of 16 bytes")

    for name in ("kvf_workspace_size", "prefill_workspace_size"):
        record(name, lambda *a: 256)
    for name in ("kvf_append", "kvf_gather", "kvf_meta_build", "kvf_paged_decode"):
        record(name)
    record("kvf_paged_prefill", prefill)
    return calls4


def _decoder(**kw):
    args = dict(batch=3, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, page_size=16, max_pages=6, num_pool_pages=14,
                max_tokens=200, device="cpu", bits=8)
    args.update(kw)
    return qskv.QuantizedPagedDecoder(**args)


def _refused_queries(n, dtype):
    """n queries of HQ heads, on the 16-byte grid, whose rows are one, overlap, or lie against one another's order."""
    x = torch.zeros((n + 1) * HQ * D, dtype=dtype)
    for stride in (0, 16, HQ * D // 2, HQ * D - 8):
        yield x.as_strided((n, HQ, D), (stride, D, 1))
    yield torch.zeros((1, HQ, D), dtype=dtype).expand(n, -1, -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top_k", [None, 2])
def test_a_refused_prefill_stores_nothing(calls, dtype, top_k):
    dec = _decoder(top_k=top_k)
    dec.prefill(torch.zeros((45, HQ, D), dtype=dtype), _tokens(45), _tokens(45), [20, 5, 20])
    before = _state(dec)
    stored = [c for c in calls if c[0] in ("extend_tables", "kvf_append", "kvf_meta_build")]
    for q in _refused_queries(7, dtype):
        with pytest.raises((ValueError, qskv.QskvError), match="q"):
            dec.prefill(q, _tokens(7), _tokens(7), [0, 3, 4])
        assert _state(dec) == before
        assert [c for c in calls if c[0] in ("extend_tables", "kvf_append", "kvf_meta_build")] == stored
    dec.prefill(torch.zeros((1, HQ, D), dtype=dtype).expand(1, -1, -1), _tokens(1), _tokens(1), [0, 0, 1])  # one row has no stride
    wide = torch.zeros((9, HQ + 2 * HKV, D), dtype=dtype)
    dec.prefill(wide[:, :HQ], wide[:, HQ:HQ + HKV], wide[:, HQ + HKV:], [0, 9, 0])
    assert dec.lengths == dec.seq_lens.tolist() == [20, 14, 21]
    assert sorted(_held(dec) + dec.free_pages.tolist()) == list(range(14))


@pytest.mark.parametrize("what,last", [("prefill", "kvf_paged_prefill"), ("step", "kvf_paged_decode"), ("step", "kvf_append"),
                                       ("prefill", "kvf_append")])
def test_a_call_that_fails_late_is_undone(calls, monkeypatch, what, last):
    """A refusal by any call of a prefill or a step leaves lengths and pages as they were, and the next one goes on from there."""
    dec = _decoder()
    q = {"prefill": torch.zeros((40, HQ, D)), "step": torch.zeros((3, HQ, D))}[what]
    dec.prefill(torch.zeros((45, HQ, D)), _tokens(45), _tokens(45), [20, 5, 20])
    before = _state(dec)
    with monkeypatch.context() as m:
        m.setattr(engine.B, last, lambda *a, **kw: (_ for _ in ()).throw(qskv.QskvError(3, "no")))
        with pytest.raises(qskv.QskvError):
            getattr(dec, what)(q, _tokens(40), _tokens(40), [0, 30, 10])
    assert _state(dec) == before
    getattr(dec, what)(q, _tokens(40), _tokens(40), [0, 30, 10])
    assert dec.lengths == dec.seq_lens.tolist() == [20, 35, 30]


def test_tokens_that_extend_made_room_for_are_still_awaited_after_a_refusal(calls):
    dec = _decoder()
    dec.extend([2, 0, 1])
    for what, q in ((dec.prefill, torch.zeros((2, HQ, D))), (dec.step, torch.zeros((3, HQ, D)))):
        with pytest.raises(ValueError, match="not stored yet"):
            what(q, _tokens(2), _tokens(2), [1, 1, 0])
    dec.append(_tokens(3), _tokens(3))
    assert dec.lengths == dec.seq_lens.tolist() == [2, 0, 1]


def test_sums_at_any_place_of_a_longer_buffer(calls):
    """lse of the prefill needs no more than its type's alignment, as the library's call has it."""
    dec = _decoder(num_q_heads=2, num_kv_heads=2)
    sums = torch.zeros((9, 2))
    for at, n in ((0, 3), (3, 2)):
        dec.prefill(torch.zeros((n, 2, D)), _tokens(n), _tokens(n), [n, 0, 0], lse=sums[at:at + n])
        assert calls[-1][0] == "kvf_paged_prefill" and calls[-1][2]["lse"].data_ptr() == sums[at:].data_ptr()
    with pytest.raises(ValueError, match="out"):
        dec.prefill(torch.zeros((2, 2, D)), _tokens(2), _tokens(2), [2, 0, 0], out=torch.zeros(2 * 2 * D + 1)[1:].view(2, 2, D))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_refused_prefill_stores_nothing_on_the_gpu(dtype):
    """A decoder that was given bad prefills between the good ones ends with the bits of one that was not."""
    from query_aware_sparse_kv_gb300 import build

    build.build()
    ends = []
    for bad in (False, True):
        g = torch.Generator().manual_seed(6)
        dec = _decoder(device="cuda", top_k=2)
        outs = []
        for new in ([25, 0, 40], [1, 7, 1], [0, 20, 3]):
            n = sum(new)
            q, k, v = (torch.randn((n, h, D), generator=g).to(dtype).cuda() for h in (HQ, HKV, HKV))
            if bad:
                at = dec.lengths, dec.free_pages.numel()
                for x in [x.cuda().as_strided(x.shape, x.stride()) for x in _refused_queries(n, dtype)] + [q[:1].expand(n, -1, -1)]:
                    with pytest.raises(ValueError, match="q"):
                        dec.prefill(x, k, v, new)
                    assert at == (dec.lengths, dec.free_pages.numel())
            outs.append(dec.prefill(q, k, v, new))
            dec.check()
        dec.step(torch.randn((3, HQ, D), generator=g).cuda(), k[:3], v[:3])
        dec.check()
        ends.append((*outs, dec.out, dec.selected, *dec.gather(0), *dec.gather(1), *dec.gather(2)))
    for x, y in zip(*ends):
        assert torch.equal(x, y)
