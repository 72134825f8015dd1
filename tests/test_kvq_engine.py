"""QuantizedPagedDecoder's own work, on the CPU: the library's calls replaced by records and 64-bit statements."""
import contextlib

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv
from query_aware_sparse_kv_gb300 import build, engine

gpu = pytest.mark.gpu


@pytest.fixture
def calls(monkeypatch):
    """The calls a decoder makes, in order: (name, device entered, stream entered, arguments)."""
    build.build()
    made, device, stream = [], [], []

    @contextlib.contextmanager
    def enter(stack, what):
        stack.append(what)
        yield
        stack.pop()

    def record(name, fn=None):
        def call(*args, **kw):
            made.append((name, device[-1] if device else None, stream[-1] if stream else None, args, kw))
            return fn(*args, **kw) if fn else None

        monkeypatch.setattr(engine.B, name, call)

    def tables(seq_lens, new_lens, free_pages, page_table, seq_lens_out, cu_new, slot_map, shape, workspace, positions,
               touched_ids, touched_valid, stream=None):
        r = R.tables(seq_lens.tolist(), new_lens.tolist(), free_pages.tolist(), page_table.tolist(), shape.page_size,
                     shape.num_pool_pages, slot_map.numel(), touched_ids.numel())
        for t, name in ((page_table, "page_table"), (seq_lens_out, "seq_lens_out"), (cu_new, "cu_new"),
                        (slot_map, "slot_map"), (positions, "positions"), (touched_ids, "touched_ids"),
                        (touched_valid, "touched_valid")):
            t.copy_(torch.tensor(r[name], dtype=torch.int32).view(t.shape))

    monkeypatch.setattr(torch.cuda, "device", lambda d: enter(device, d))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: enter(stream, s))
    for name in ("kvq_workspace_size", "tables_workspace_size", "workspace_size"):
        record(name, lambda shape: 256)
    record("extend_tables", tables)
    record("get_error", lambda *a: 0)
    for name in ("kvq_append", "kvq_gather", "kvq_meta_build", "page_select", "kvq_paged_decode"):
        record(name)
    return made


def _decoder(**kw):
    args = dict(batch=3, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, max_pages=6, num_pool_pages=14,
                max_tokens=200, device="cpu")
    args.update(kw)
    return qskv.QuantizedPagedDecoder(**args)


def _tokens(n, hkv=2, d=64):
    return torch.zeros((n, hkv, d))


def _held(dec):
    return [int(p) for b, n in enumerate(dec.lengths) for p in dec.page_table[b, :-(-n // 16)]]


def test_free_pages_stay_in_one_buffer(calls):
    """Pages given back and taken again, in many orders: always each page once, and always in the storage the decoder
    began with (none goes back to the allocator while another stream may read it)."""
    dec = _decoder()
    g = torch.Generator().manual_seed(0)
    at = dec.free_pages.untyped_storage().data_ptr()
    for _ in range(200):
        row = int(torch.randint(0, 3, (1,), generator=g))
        if torch.rand((), generator=g) < 0.4:
            dec.release(row)
            assert dec.lengths[row] == 0 and int(dec.seq_lens[row]) == 0
        else:
            new = [0, 0, 0]
            new[row] = min(int(torch.randint(0, 60, (1,), generator=g)), 96 - dec.lengths[row])
            before = list(dec.lengths)
            try:
                dec.extend(new)
            except ValueError:
                assert dec.lengths == before
                continue
            dec.append(_tokens(sum(new)), _tokens(sum(new)))
        assert dec.seq_lens.tolist() == dec.lengths
        assert sorted(_held(dec) + dec.free_pages.tolist()) == list(range(14))
        assert dec.free_pages.untyped_storage().data_ptr() == at


def test_calls_without_a_device_of_their_own_run_on_the_decoders(calls):
    """The selection and the error check go to the current device: the decoder makes its own that."""
    dec = _decoder(top_k=2)
    dec.step(torch.zeros((3, 4, 64)), _tokens(5), _tokens(5), [2, 0, 3])
    dec.check()
    entered = {name: device for name, device, *_ in calls}
    for name in ("workspace_size", "kvq_workspace_size", "tables_workspace_size", "page_select", "get_error"):
        assert entered[name] == dec.pool.device, name


def test_raw_stream_handles(calls, monkeypatch):
    """A stream as a number, as every call of the library takes it: torch's own work goes to that stream too."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    dec = _decoder()
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s) or contextlib.nullcontext())
    for handle, want in ((0x7100, ("external", 0x7100, dec.pool.device)), (0, ("default", dec.pool.device)), (None, None)):
        del calls[:], entered[:]
        dec.step(torch.zeros((3, 4, 64)), _tokens(5), _tokens(5), [2, 0, 3], stream=handle)
        dec.gather(2, stream=handle)
        dec.release(2, stream=handle)
        assert entered == [want] * 3
        for name, _, _, args, kw in calls:
            assert kw.get("stream", args[-1]) == handle, name


def _bad_queries(dtype=torch.float32):
    """Queries that a decoder of 3 rows, 4 heads of 64 dims refuses."""
    flat = torch.zeros(3 * 4 * 64 + 1, dtype=dtype)
    yield torch.zeros((2, 4, 64), dtype=dtype)  # not every row's
    yield torch.zeros((3, 2, 64), dtype=dtype)
    yield torch.zeros((3, 4, 128), dtype=dtype)
    yield torch.zeros((3, 4, 64), dtype=torch.float16)
    yield torch.zeros((3, 64, 4), dtype=dtype).transpose(1, 2)
    yield flat[1:].view(3, 4, 64)  # not on 16 bytes


def test_the_selection_is_given_queries_of_every_row_only(calls):
    """page_select is handed an address: shorter queries would be read past their end."""
    dec = _decoder(top_k=2)
    for q in _bad_queries():
        with pytest.raises((ValueError, TypeError)):
            dec.select(q)
    assert "page_select" not in [c[0] for c in calls]
    dec.select(torch.zeros((3, 4, 64), dtype=torch.bfloat16))
    assert calls[-1][0] == "page_select"


def _state(dec):
    return (list(dec.lengths), dec.seq_lens.tolist(), dec.free_pages.tolist(),
            [dec.page_table[b, :-(-n // 16)].tolist() for b, n in enumerate(dec.lengths)])


def test_a_refused_step_changes_nothing(calls, monkeypatch):
    dec = _decoder()
    q = torch.zeros((3, 4, 64))
    dec.step(q, _tokens(45), _tokens(45), [20, 5, 20])
    before = _state(dec)
    stored = len([c for c in calls if c[0] == "kvq_append"])
    for bad in _bad_queries():
        with pytest.raises((ValueError, TypeError)):
            dec.step(bad, _tokens(3), _tokens(3))
    for k, new in ((_tokens(2), None), (_tokens(4), None), (_tokens(3), [1, 1]), (_tokens(3), [-1, 1, 3]), (None, None),
                   (_tokens(100), [100, 0, 0])):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            dec.step(q, k, k, new)
    with monkeypatch.context() as m:  # a refusal by the call that stores
        m.setattr(engine.B, "kvq_append", lambda *a: (_ for _ in ()).throw(ValueError("k must be ..")))
        with pytest.raises(ValueError, match="k must be"):
            dec.step(q, _tokens(40), _tokens(40), [0, 30, 10])
    assert _state(dec) == before and len([c for c in calls if c[0] == "kvq_append"]) == stored
    dec.step(q, _tokens(40), _tokens(40), [0, 30, 10])
    assert dec.lengths == dec.seq_lens.tolist() == [20, 35, 30]
    assert sorted(_held(dec) + dec.free_pages.tolist()) == list(range(14))


def test_arguments_that_no_step_could_run_with(calls):
    """Refused when the decoder is made, not by a step that has stored its tokens."""
    for bad in (dict(top_k=0), dict(top_k=-3), dict(max_tokens=0), dict(sm_scale=-1.0), dict(sm_scale=float("nan")),
                dict(sm_scale=float("inf"))):
        with pytest.raises(ValueError, match=list(bad)[0]):
            _decoder(**bad)
    for bad in (dict(group_size=48), dict(head_dim=96), dict(page_size=24), dict(batch=0), dict(num_q_heads=6)):
        with pytest.raises(qskv.QskvError):
            _decoder(**bad)
    with pytest.raises(ValueError, match="selects none"):
        _decoder(top_k=None).select(torch.zeros((3, 4, 64)))


@gpu
def test_pages_given_back_on_a_stream_that_is_behind():
    """release on a stream with work before it; other tensors of the list's size are made and filled on the default stream
    meanwhile, and the pages handed out afterwards are still each another one."""
    build.build()
    dec = _decoder(batch=40, max_pages=2, num_pool_pages=70, device="cuda")
    k = torch.zeros((35 * 20, 2, 64), device="cuda")
    x = torch.randn((2048, 2048), device="cuda")
    side = torch.cuda.Stream()
    for rows in range(0, 35, 5):
        new = [20 if rows <= b < rows + 5 else 0 for b in range(40)]
        dec.extend(new)
        dec.append(k[:100], k[:100])
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                x = x @ x * 1e-3
        for b in range(5, 10):
            dec.release(b, stream=side)
            fill = [torch.full((n,), -5, dtype=torch.int32, device="cuda") for n in (2, 10, 60, 62, 64, 66, 70, 128)]
        torch.cuda.current_stream().wait_stream(side)
        assert sorted(_held(dec) + dec.free_pages.tolist()) == list(range(70))
        dec.extend([20 if 5 <= b < 10 else 0 for b in range(40)])
        dec.append(k[:100], k[:100])
        dec.check()
        assert sorted(_held(dec) + dec.free_pages.tolist()) == list(range(70)) and len(fill) == 8


@gpu
def test_raw_stream_handles_on_the_gpu():
    build.build()
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((40, 2, 64), generator=g).cuda() for _ in range(2))
    q = torch.randn((3, 4, 64), generator=g).cuda()
    side, outs = torch.cuda.Stream(), []
    for stream in (None, side, side.cuda_stream, 0):
        torch.cuda.synchronize()
        dec = _decoder(device="cuda", top_k=2)
        torch.cuda.synchronize()
        dec.step(q, k, v, [25, 0, 15], stream=stream)
        dec.release(0, stream=stream)
        dec.step(q, k[:20], v[:20], [18, 0, 2], stream=stream)
        got = dec.gather(0, stream=stream)
        dec.check(stream=stream)
        torch.cuda.synchronize()
        outs.append((dec.out, dec.lse, *got))
    for other in outs[1:]:
        for x, y in zip(outs[0], other):
            assert torch.equal(x, y)


@gpu
@pytest.mark.parametrize("top_k", [None, 2])
def test_a_refused_step_changes_nothing_on_the_gpu(top_k):
    """A decoder that was given bad steps between the good ones ends with the bits of one that was not."""
    build.build()
    outs = []
    for bad in (False, True):
        g = torch.Generator().manual_seed(4)
        dec = _decoder(device="cuda", top_k=top_k)
        for new in ([25, 0, 40], [1, 1, 1], [1, 17, 1]):
            k, v = (torch.randn((sum(new), 2, 64), generator=g).cuda() for _ in range(2))
            q = torch.randn((3, 4, 64), generator=g).cuda()
            if bad:
                for args in ((q[:2], k, v, new), (q.half(), k, v, new), (q, k.half(), v.half(), new), (q, k, v[:1], new),
                             (q, k[:1], v[:1], new), (q, k.cpu(), v, new), (q, k[:, :1], v[:, :1], new),
                             (q, k, v, [n + 200 for n in new]), (q.cpu(), k, v, new),
                             (q, k.transpose(1, 2).contiguous().transpose(1, 2), v, new)):
                    with pytest.raises((ValueError, TypeError)):
                        dec.step(*args)
            dec.step(q, k, v, new)
            dec.check()
        outs.append((dec.out, dec.lse, *dec.gather(0), *dec.gather(2)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
