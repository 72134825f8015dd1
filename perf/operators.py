"""Cases of the 4-bit paged KV cache operators: what is timed, and their plain forms.

Operators (q query heads, Hkv KV heads, d = head_dim, P = page_size, gs = group size, NG = d / gs):

  tables   qskv.extend_tables      page tables, slot map, positions and touched-page list of one
                                   scheduler step, from the requests' lengths and a list of free pages
  append   qskv.kvq_append         new tokens' keys and values quantised to 4 bits and stored by slot
  gather   qskv.kvq_gather         cached tokens read back as values, by slot
  meta     qskv.kvq_meta_build     element-wise min / max of a page's cached keys (bf16, rounded outwards)
  decode   qskv.kvq_paged_decode   attention of one query token a sequence over its cached pages, all of
                                   them or a selected list

Numbers held in 4 bits.  A group of gs neighbouring dims of one token and head, x_0..x_{gs-1}, is stored as
    m  = bf16(min x)                      (round to nearest even)
    s  = bf16((max x - m) / 15)           (one rounding; 0 if not at least 2^-100)
    u  = clamp(rint((x - m) / s), 0, 15)  (ties to even; 0 if s = 0)
and stands for m + s u.

One (page, head) block of the pool, in 32-bit words (little endian), P tokens, W = d / 8 words a token:
    [P][W] key codes | [P][W] value codes | [NG][P] key params | [NG][P] value params
Code word w of a token holds dims 8w..8w+7, dim 8w+k in bits 4k..4k+3.  A key's word w = 4i + t is stored at
place t * (d / 32) + i of its row; a value's word w = 4c + j of token t at place 4 (c ^ x) + j, with
x = (t / 2) % 4 for d = 128 and (t / 4) % 2 for d = 64.  A param word is bf16 s in the low half, bf16 m in the high.
"""
import math

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634


def _qskv():
    import query_aware_sparse_kv_gb300 as qskv

    return qskv


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one scheduler step of a decode batch: one new token a request
        dict(name="tables_decode_256", op="tables", batch=256, page=16, max_pages=2048, max_tokens=256, lo=1, hi=32000,
             new="one"),
        # admission of many requests with prompts of mixed length beside running ones
        dict(name="tables_mixed_1500", op="tables", batch=1500, page=16, max_pages=2048, max_tokens=400_000, lo=0,
             hi=8192, new="mixed"),
        # a decode step's tokens, one a sequence
        dict(name="append_decode_32", op="append", tokens=32, hq=32, hkv=8, d=128, page=16, gs=128, dtype="bf16",
             kind="decode"),
        # a prefill step's tokens, taken as views of the fused projection's output
        dict(name="append_prefill_32k", op="append", tokens=32_768, hq=32, hkv=8, d=128, page=16, gs=64, dtype="bf16",
             kind="prefill"),
        # a short context read back (a prefix moved to another cache)
        dict(name="gather_short_257", op="gather", tokens=257, hkv=16, d=64, page=16, gs=64, dtype="fp32"),
        # a long context read back for a chunk's prefill attention
        dict(name="gather_context_131k", op="gather", tokens=131_072, hkv=8, d=128, page=32, gs=32, dtype="bf16"),
        # the pages that a decode batch appends to
        dict(name="meta_last_pages_32", op="meta", pages=32, pool=2048, hkv=8, d=128, page=16, gs=128),
        # every page of a batch after prefill
        dict(name="meta_prefill_36864", op="meta", pages=36_864, pool=36_900, hkv=8, d=128, page=16, gs=64),
        # the smallest decode: two short sequences, where latency counts
        dict(name="decode_tiny_fp32", op="decode", batch=2, hq=4, hkv=2, d=64, page=16, gs=64, lo=1, hi=256, top_k=0,
             dtype="fp32"),
        # the headline batch: 128 selected pages of 4K..32K tokens
        dict(name="decode_gqa4_top128", op="decode", batch=32, hq=32, hkv=8, d=128, page=16, gs=128, lo=4096,
             hi=32_768, top_k=128, dtype="bf16"),
        # a ragged serving batch with 8 query heads a KV head, empty rows among them, all pages
        dict(name="decode_gqa8_ragged", op="decode", batch=64, hq=64, hkv=8, d=128, page=16, gs=64, lo=0, hi=4095,
             top_k=0, dtype="fp32"),
        # long contexts, all pages
        dict(name="decode_long_dense", op="decode", batch=4, hq=32, hkv=8, d=128, page=32, gs=32, lo=65_536,
             hi=131_072, top_k=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "gather", "meta", "decode", "decode"])
    page = rng.choice([16, 32])
    if op == "tables":
        batch = _log(rng, 1, 4000)
        if rng.random() < 0.5:
            return dict(op=op, batch=batch, page=page, max_pages=2048, max_tokens=batch + rng.randrange(0, 9), lo=0,
                        hi=_log(rng, 16, 32_000), new="one")
        return dict(op=op, batch=batch, page=page, max_pages=1024, max_tokens=_log(rng, max(64, 8 * batch), 400_000), lo=0,
                    hi=_log(rng, 16, 8192), new="mixed")
    d = rng.choice([64, 128])
    gs = rng.choice([g for g in (32, 64, 128) if g <= d])
    hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        kind = rng.choice(["decode", "prefill"])
        tokens = _log(rng, 1, 600) if kind == "decode" else _log(rng, 17, 262_144 // hkv)
        return dict(op=op, tokens=tokens, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=d, page=page, gs=gs,
                    dtype=rng.choice(["bf16", "fp32"]), kind=kind)
    if op == "gather":
        return dict(op=op, tokens=_log(rng, 1, 1_000_000 // hkv), hkv=hkv, d=d, page=page, gs=gs,
                    dtype=rng.choice(["bf16", "fp32"]))
    if op == "meta":
        pages = _log(rng, 1, 290_000 // hkv // (page // 16))
        return dict(op=op, pages=pages, pool=pages + rng.randrange(1, 100), hkv=hkv, d=d, page=page, gs=gs)
    group = rng.choice([1, 2, 4, 8])
    batch = _log(rng, 1, 256)
    hi = _log(rng, 1, min(131_072, max(1, 2_000_000 // (batch * hkv))))
    return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page, gs=gs, lo=rng.choice([0, 1, hi // 2]),
                hi=hi, top_k=rng.choice([0, 0, 1, 7, 32, 128]), dtype=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------- the cache's format --
def _block_words(c):
    return (c["page"] * c["d"] + 8 * c["page"] * (c["d"] // c["gs"])) // 4


def _key_places(d, dev):
    """Place of each of a key's code words in its row."""
    w = torch.arange(d // 8, device=dev)
    return (w % 4) * (d // 32) + w // 4


def _value_places(d, page, dev):
    """Place of each of a value's code words in its row, for every token of a page."""
    w = torch.arange(d // 8, device=dev)[None, :]
    t = torch.arange(page, device=dev)[:, None]
    x = (t // 2) % 4 if d == 128 else (t // 4) % 2
    return 4 * ((w // 4) ^ x) + w % 4


def _bf16_once(x):
    """Doubles >= 0 rounded to bf16 once (through fp32 rounded to odd, so that no second rounding shows)."""
    f = x.float()
    bits = f.view(torch.int32)
    bits = torch.where(f.double() > x, bits - 1, bits)  # towards zero
    inexact = (bits.view(torch.float32).double() != x) & torch.isfinite(f)
    return (bits | inexact.int()).view(torch.float32).to(torch.bfloat16)


def _quantise(x, gs):
    """x [..., d] -> codes int32 [..., d], s and m bf16 [..., d / gs]."""
    g = x.unflatten(-1, (-1, gs))
    m = g.amin(-1).to(torch.bfloat16)
    step = (g.amax(-1).double() - m.double()) / 15
    s = torch.where(step >= 2.0 ** -100, _bf16_once(step.clamp_min(0)), torch.zeros_like(m))
    one = torch.where(s > 0, s.double(), torch.ones_like(step))
    u = torch.round((g.double() - m.double()[..., None]) / one[..., None]).clamp_(0, 15)
    u = torch.where((s > 0)[..., None], u, torch.zeros_like(u))
    return u.to(torch.int32).flatten(-2), s, m


def _words(codes):
    """Codes [..., d] -> 32-bit words [..., d / 8]."""
    sh = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    return (codes.unflatten(-1, (-1, 8)) << sh).sum(-1).to(torch.int32)


def _params(s, m):
    return (s.view(torch.int16).to(torch.int32) & 0xFFFF) | (m.view(torch.int16).to(torch.int32) << 16)


def _store(c, pool, slots, k, v):
    """Tokens k, v [n][Hkv][d] into the slots of pool [Npool][Hkv][words] (int32 words)."""
    d, P, gs, H = c["d"], c["page"], c["gs"], c["hkv"]
    W, NG = d // 8, d // gs
    # a negative slot repeats the first token's store
    keep = torch.where(slots >= 0, torch.arange(len(slots), device=slots.device), 0)
    slot = slots[keep].long()
    base = (slot // P * H)[:, None] + torch.arange(H, device=slot.device)
    base, t = base * _block_words(c), slot % P
    flat = pool.view(-1)
    row = base + (t * W)[:, None]
    col = torch.arange(NG, device=slot.device) * P
    for at, x, params in ((None, k, 2 * P * W), (P * W, v, 2 * P * W + NG * P)):
        codes, s, m = _quantise(x[keep], gs)
        if at is None:
            place = row[:, :, None] + _key_places(d, slot.device)
        else:
            place = (row + at)[:, :, None] + _value_places(d, P, slot.device)[t][:, None, :]
        flat[place] = _words(codes)
        flat[(base + t[:, None])[:, :, None] + params + col] = _params(s, m)


def _unpack(c, words, which):
    """Blocks' words [..., block words] -> values fp32 [..., P, d] of the keys (0) or the values (1)."""
    d, P, NG = c["d"], c["page"], c["d"] // c["gs"]
    W = d // 8
    dev = words.device
    at = _value_places(d, P, dev) + P * W if which else _key_places(d, dev)[None, :]
    w = words[..., torch.arange(P, device=dev)[:, None] * W + at]  # [..., P, W]
    sh = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    u = ((w[..., None] >> sh) & 15).flatten(-2).float()
    p0 = 2 * P * W + which * NG * P
    p = words[..., p0:p0 + NG * P].unflatten(-1, (NG, P)).transpose(-1, -2)  # [..., P, NG]
    s, m = (p << 16).view(torch.float32), (p & -65536).view(torch.float32)
    return (m[..., None] + s[..., None] * u.unflatten(-1, (NG, -1))).flatten(-2)


def _read(c, pool, slots, which, dtype):
    """Values [n][Hkv][d] of the slots (0 where a slot is negative)."""
    P, H, d = c["page"], c["hkv"], c["d"]
    W, NG = d // 8, d // c["gs"]
    slot = slots.clamp_min(0).long()
    base = ((slot // P * H)[:, None] + torch.arange(H, device=slot.device)) * _block_words(c)
    t = slot % P
    if which:
        place = (base + (P * W + t * W)[:, None])[:, :, None] + _value_places(d, P, slot.device)[t][:, None, :]
    else:
        place = (base + (t * W)[:, None])[:, :, None] + _key_places(d, slot.device)
    flat = pool.view(-1)
    sh = torch.arange(0, 32, 4, device=slot.device, dtype=torch.int32)
    u = ((flat[place][..., None] >> sh) & 15).flatten(-2).float()
    p0 = 2 * P * W + which * NG * P
    p = flat[(base + t[:, None])[:, :, None] + p0 + torch.arange(NG, device=slot.device) * P]
    s, m = (p << 16).view(torch.float32), (p & -65536).view(torch.float32)
    x = (m[..., None] + s[..., None] * u.unflatten(-1, (NG, -1))).flatten(-2)
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(dtype)


def _towards(x, up):
    """fp32 -> bf16, rounded up or down."""
    b = x.to(torch.bfloat16)
    far = b.float() < x if up else b.float() > x
    bits = b.view(torch.int16).to(torch.int32)
    # the neighbour above (below): away from zero for a value of that sign, towards it for the other
    away = (bits >= 0) if up else (bits < 0)
    moved = torch.where(away, bits + 1, bits - 1)
    if up:
        moved = torch.where(bits == -32768, torch.ones_like(bits), moved)
    else:
        moved = torch.where(bits == 0, torch.full_like(bits, -32767), moved)
    return torch.where(far, moved, bits).to(torch.int16).view(torch.bfloat16)


# ------------------------------------------------------------------ inputs --
def _dtype(c):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[c["dtype"]]


def _shape_of(c, batch, hq, max_pages, pool):
    return _qskv().make_shape(batch, hq, c["hkv"], c["d"], c["page"], max_pages, pool)


def _keys(g, *shape):
    """Keys or values as projections make them: some dims with an offset and a larger spread."""
    d = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda")
    spread = 0.5 + torch.rand(d, generator=g, device="cuda")
    return x * spread + 2.0 * torch.randn(d, generator=g, device="cuda") * (torch.rand(d, generator=g, device="cuda") < 0.1)


def _pool(c, g, pages):
    """A pool of `pages` pages of quantised keys and values."""
    d, P, H, gs = c["d"], c["page"], c["hkv"], c["gs"]
    W, NG = d // 8, d // gs
    pool = torch.empty((pages, H, _block_words(c)), dtype=torch.int32, device="cuda")
    step = max(1, (1 << 25) // (P * H * d))
    vp = _value_places(d, P, pool.device)
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for which in (0, 1):
            codes, s, m = _quantise(_keys(g, n, H, P, d), gs)
            w = _words(codes)
            to = pool[a:a + n, :, which * P * W:(which + 1) * P * W].view(n, H, P, W)
            if which:
                to.scatter_(3, vp.expand(n, H, P, W), w)
            else:
                to[..., _key_places(d, pool.device)] = w
            p0 = 2 * P * W + which * NG * P
            pool[a:a + n, :, p0:p0 + NG * P] = _params(s, m).transpose(-1, -2).flatten(-2)
    return pool


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    P = c["page"]
    ints = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] == "tables":
        B, mp = c["batch"], c["max_pages"]
        old = ints(min(c["lo"], c["hi"]), c["hi"], B)
        if c["new"] == "one":
            new = torch.ones(B, dtype=torch.int64, device="cuda")
        else:  # two in three requests run on by a token, the others bring a prompt; what fits max_tokens
            prompt = torch.rand(B, generator=g, device="cuda") < 1 / 3
            most = max(1, int(1.5 * c["max_tokens"] / B))
            new = torch.where(prompt, ints(1, most, B), torch.ones_like(old))
            old = torch.where(prompt & (torch.rand(B, generator=g, device="cuda") < 0.7), torch.zeros_like(old), old)
        old = torch.minimum(old, mp * P - new.clamp(max=mp * P))
        new = torch.minimum(new, mp * P - old)
        new = torch.where(torch.cumsum(new, 0) <= c["max_tokens"], new, torch.zeros_like(new))
        have = (old + P - 1) // P
        need = (old + new + P - 1) // P - have
        pool = int(have.sum() + need.sum()) + 37
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        j = torch.arange(mp, device="cuda")[None, :]
        start = (torch.cumsum(have, 0) - have)[:, None]
        table = torch.where(j < have[:, None], ids[(start + j).clamp(max=pool - 1)], torch.full_like(ids[:1], -1))
        cap = min(c["max_tokens"], c["max_tokens"] // P + 2 * B)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        st.update(seq_lens=old.to(torch.int32), new_lens=new.to(torch.int32), free_pages=ids[int(have.sum()):].clone(),
                  page_table=table.contiguous(), seq_lens_out=i32(B), cu_new=i32(B + 1), slot_map=i32(c["max_tokens"]),
                  positions=i32(c["max_tokens"]), touched_ids=i32(cap), touched_valid=i32(cap), counts=i32(4))
        if own:
            st["shape"] = _qskv().make_shape(B, 8, 8, 128, P, mp, pool)
    elif c["op"] in ("append", "gather"):
        n, H, d = c["tokens"], c["hkv"], c["d"]
        if c.get("kind") == "decode":  # each token in a page of its own, anywhere in it
            pages = n + 13
            slots = torch.randperm(pages, generator=g, device="cuda")[:n] * P + ints(0, P - 1, n)
        else:  # runs of up to about 1000 tokens, each in pages of its own; a few padded places at the end
            length = min(n, 1000) if n > 40 else n
            runs = -(-n // length)
            per = -(-(length + P) // P)
            pages = runs * per + 13
            i = torch.arange(n, device="cuda")
            at = i % length + ints(0, P - 1, runs)[i // length]
            slots = torch.randperm(pages, generator=g, device="cuda")[i // length * per + at // P] * P + at % P
            slots[n - n // 50:] = -1
        st["slots"] = slots.to(torch.int32)
        st["k_out"] = torch.empty((n, H, d), dtype=_dtype(c), device="cuda")
        st["v_out"] = torch.empty((n, H, d), dtype=_dtype(c), device="cuda")
        if c["op"] == "append":
            qkv = torch.cat([torch.randn((n, c["hq"], d), generator=g, device="cuda"), _keys(g, n, H, d),
                             _keys(g, n, H, d)], 1).to(_dtype(c))
            st["k"], st["v"] = qkv[:, c["hq"]:c["hq"] + H], qkv[:, c["hq"] + H:]
            st["pool"] = torch.zeros((pages, H, _block_words(c)), dtype=torch.int32, device="cuda")
        else:
            st["pool"] = _pool(c, g, pages)
        if own:
            st["shape"] = _shape_of(c, 1, c.get("hq", H), 1, pages)
    elif c["op"] == "meta":
        st["pool"] = _pool(c, g, c["pool"])
        st["page_ids"] = torch.randperm(c["pool"], generator=g, device="cuda")[:c["pages"]].to(torch.int32)
        st["valid"] = torch.where(torch.rand(c["pages"], generator=g, device="cuda") < 0.1, ints(1, P, c["pages"]),
                                  torch.full((c["pages"],), P, device="cuda")).to(torch.int32)
        st["meta"] = torch.zeros((c["pool"], c["hkv"], 2, c["d"]), dtype=torch.bfloat16, device="cuda")
        if own:
            st["shape"] = _shape_of(c, 1, c["hkv"], 1, c["pool"])
    else:
        B, H, d = c["batch"], c["hkv"], c["d"]
        lens = ints(min(c["lo"], c["hi"]), c["hi"], B)
        n = (lens + P - 1) // P
        mp, total = max(1, -(-c["hi"] // P)), int(n.sum())
        pool = total + 5
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        j = torch.arange(mp, device="cuda")[None, :]
        start = (torch.cumsum(n, 0) - n)[:, None]
        table = torch.where(j < n[:, None], ids[(start + j).clamp(max=pool - 1)], torch.full_like(ids[:1], -1))
        st.update(pool=_pool(c, g, pool), page_table=table.contiguous(), seq_lens=lens.to(torch.int32))
        # slots past a sequence's end hold whatever was there before
        last = torch.nonzero(lens % P).flatten()
        if len(last):
            page = table[last, n[last] - 1].long()
            W, NG = d // 8, d // c["gs"]
            t = torch.arange(P, device="cuda")[None, :] >= (lens[last] % P)[:, None]
            bad = st["pool"][page][:, :, 2 * P * W:].unflatten(-1, (2 * NG, P))
            bad = torch.where(t[:, None, None, :], torch.full_like(bad, 0x7FC07FC0), bad)
            st["pool"][page[:, None], :, torch.arange(2 * P * W, _block_words(c), device="cuda")[None, :]] = \
                bad.flatten(-2).transpose(1, 2)
        st["q"] = torch.randn((B, c["hq"], d), generator=g, device="cuda").to(_dtype(c))
        st["out"] = torch.empty((B, c["hq"], d), device="cuda")
        st["lse"] = torch.empty((B, c["hq"]), device="cuda")
        if c["top_k"]:
            K = c["top_k"]
            key = torch.rand((B, H, mp), generator=g, device="cuda").masked_fill_((j >= n[:, None])[:, None, :], 2.0)
            pick = key.argsort(-1)[..., :K].to(torch.int32)
            pick = torch.where(torch.arange(pick.shape[-1], device="cuda") < n[:, None, None], pick,
                               torch.full_like(pick, 1 << 30)).sort(-1).values
            pick = torch.where(pick == 1 << 30, torch.full_like(pick, -1), pick)
            st["selected"] = torch.nn.functional.pad(pick, (0, K - pick.shape[-1]), value=-1).contiguous()
            st["n_selected"] = n.clamp(max=K).to(torch.int32)[:, None].expand(B, H).contiguous()
        if own:
            st["shape"] = _shape_of(c, B, c["hq"], mp, pool)
    if "pool" in st:  # the cache as a user holds it: bytes
        st["pool"] = st["pool"].view(torch.uint8)
    if own:
        size = _qskv().kvq_workspace_size(st["shape"]) if c["op"] == "decode" else 256
        if c["op"] == "tables":
            size = _qskv().tables_workspace_size(st["shape"])
        st["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------- one pass --
def run(st):
    return globals()["_run_" + st["case"]["op"]](st)


TABLE_OUTPUTS = ("page_table", "seq_lens_out", "cu_new", "slot_map", "positions", "touched_ids", "touched_valid",
                 "counts")


def _run_tables(st):
    if own:
        _qskv().extend_tables(st["seq_lens"], st["new_lens"], st["free_pages"], st["page_table"], st["seq_lens_out"],
                              st["cu_new"], st["slot_map"], st["shape"], st["workspace"], positions=st["positions"],
                              touched_ids=st["touched_ids"], touched_valid=st["touched_valid"], counts=st["counts"])
        return {k: st[k] for k in TABLE_OUTPUTS}
    c, table, free = st["case"], st["page_table"], st["free_pages"]
    P, dev = c["page"], table.device
    old, new = st["seq_lens"].long(), st["new_lens"].long()
    have, now = (old + P - 1) // P, (old + new + P - 1) // P
    need_end, tok_end = torch.cumsum(now - have, 0), torch.cumsum(new, 0)
    ok = (new > 0) & (need_end <= free.numel()) & (tok_end <= c["max_tokens"])
    # pages taken from the free list, in order of requests
    j = torch.arange(c["max_pages"], device=dev)[None, :]
    fresh = (j >= have[:, None]) & (j < now[:, None]) & ok[:, None]
    taken = ((need_end - now)[:, None] + j).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[taken], table))
    first = old // P
    touch = torch.where(ok, now - first, torch.zeros_like(now))
    touch_end = torch.cumsum(touch, 0)
    # the touched pages, by request and place
    e = torch.arange(st["touched_ids"].numel(), device=dev)
    r = torch.searchsorted(touch_end, e, right=True)
    there = r < c["batch"]
    r = r.clamp(max=c["batch"] - 1)
    page = first[r] + e - (touch_end - touch)[r]
    page = torch.where(there, page, torch.zeros_like(page))
    ids = table[r, page]
    none = torch.full_like(ids, -1)
    touched_ids = torch.where(there, ids, none)
    valid = torch.minimum(torch.full_like(page, P), (old + new)[r] - page * P)
    touched_valid = torch.where(there, valid, torch.zeros_like(valid)).to(torch.int32)
    # the tokens
    e = torch.arange(c["max_tokens"], device=dev)
    r = torch.searchsorted(tok_end, e, right=True)
    there = r < c["batch"]
    r = r.clamp(max=c["batch"] - 1)
    there &= ok[r]
    pos = torch.where(there, old[r] + e - (tok_end - new)[r], torch.zeros_like(e))
    slot = table[r, pos // P].long() * P + pos % P
    minus = torch.full_like(slot, -1)
    cu = torch.cat([torch.zeros_like(tok_end[:1]), tok_end]).clamp(max=c["max_tokens"])
    counts = torch.stack([cu[-1], torch.where(ok, now - have, torch.zeros_like(now)).sum(), touch_end[-1],
                          ((new > 0) & ~ok).sum()])
    return dict(page_table=table, seq_lens_out=(old + torch.where(ok, new, torch.zeros_like(new))).to(torch.int32),
                cu_new=cu.to(torch.int32), slot_map=torch.where(there, slot, minus).to(torch.int32),
                positions=torch.where(there, pos, minus).to(torch.int32), touched_ids=touched_ids,
                touched_valid=touched_valid, counts=counts.to(torch.int32))


def _run_append(st):
    """Tokens stored, and read back as the values that the cache then stands for."""
    c = st["case"]
    if own:
        _qskv().kvq_append(st["k"], st["v"], st["slots"], st["pool"], st["shape"], c["gs"], st["workspace"])
        _qskv().kvq_gather(st["pool"], st["slots"], st["k_out"], st["v_out"], st["shape"], c["gs"], st["workspace"])
        return {"k": st["k_out"], "v": st["v_out"]}
    _store(c, st["pool"].view(torch.int32), st["slots"], st["k"], st["v"])
    return _run_gather(st)


def _run_gather(st):
    c = st["case"]
    if own:
        _qskv().kvq_gather(st["pool"], st["slots"], st["k_out"], st["v_out"], st["shape"], c["gs"], st["workspace"])
        return {"k": st["k_out"], "v": st["v_out"]}
    pool = st["pool"].view(torch.int32)
    return {"k": _read(c, pool, st["slots"], 0, _dtype(c)), "v": _read(c, pool, st["slots"], 1, _dtype(c))}


def _run_meta(st):
    c = st["case"]
    if own:
        _qskv().kvq_meta_build(st["pool"], st["page_ids"], st["valid"], st["meta"], st["shape"], c["gs"],
                               st["workspace"])
        return {"meta": st["meta"]}
    ids = st["page_ids"].long()
    k = _unpack(c, st["pool"].view(torch.int32)[ids], 0)  # [n][Hkv][P][d]
    off = (torch.arange(c["page"], device=ids.device) >= st["valid"][:, None])[:, None, :, None]
    st["meta"][ids] = torch.stack([_towards(k.masked_fill(off, math.inf).amin(2), False),
                                   _towards(k.masked_fill(off, -math.inf).amax(2), True)], 2)
    return {"meta": st["meta"]}


def _run_decode(st):
    c = st["case"]
    if own:
        _qskv().kvq_paged_decode(st["q"], st["pool"], st["page_table"], st["seq_lens"], st["out"], st["shape"], c["gs"],
                                 st["workspace"], selected=st.get("selected"), n_selected=st.get("n_selected"),
                                 top_k=c["top_k"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    B, H, d, P = c["batch"], c["hkv"], c["d"], c["page"]
    G = c["hq"] // H
    lens, table = st["seq_lens"].long(), st["page_table"]
    if c["top_k"]:
        sel = st["selected"].long()
        off = torch.arange(sel.shape[-1], device=sel.device) >= st["n_selected"][..., None]
        page = table[:, None, :].expand(B, H, -1).gather(2, sel.clamp_min(0)).long()
        pos = sel[..., None] * P + torch.arange(P, device=sel.device)
        off = off[..., None] | (pos >= lens[:, None, None, None])
    else:
        page = table[:, None, :].long()
        pos = torch.arange(table.shape[1] * P, device=table.device).view(1, 1, -1, P)
        off = pos >= lens[:, None, None, None]
    off = off.flatten(2)[:, :, None, :]  # [B][1 or H][1][tokens]
    blocks = st["pool"].view(torch.int32)[page.clamp_min(0), torch.arange(H, device=table.device)[None, :, None]]
    q = st["q"].float().view(B, H, G, d)
    k = _unpack(c, blocks, 0).flatten(2, 3)  # [B][H][tokens][d]
    x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    del k
    x = x.masked_fill(off, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    v = _unpack(c, blocks, 1).flatten(2, 3).masked_fill_(off.transpose(-1, -2), 0.0)
    o = (p @ v) / total.clamp_min(1e-30)
    return {"out": o.view(B, c["hq"], d), "lse": (top + torch.log(total)).view(B, c["hq"])}


# -------------------------------------------------- what a pass cannot avoid --
def work(case):
    c = case
    P = c["page"]
    if c["op"] == "tables":
        B, T = c["batch"], c["max_tokens"]
        # lengths in and out, the slot and position of each token, each touched page read or taken and written
        touched = B if c["new"] == "one" else B + T // P
        return {"bytes": 4 * (2 * B + 2 * B + 1 + 2 * T + 4 * touched), "flops": 0}
    d, H = c["d"], c["hkv"]
    cached = d + 8 * (d // c["gs"])  # bytes of one token and head, keys and values
    es = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "append":
        n = c["tokens"]
        return {"bytes": n * H * (2 * d * es + 2 * cached + 2 * d * es) + 8 * n, "flops": 8 * n * H * 2 * d}
    if c["op"] == "gather":
        n = c["tokens"]
        return {"bytes": n * H * (cached + 2 * d * es) + 4 * n, "flops": 4 * n * H * d}
    if c["op"] == "meta":
        return {"bytes": c["pages"] * (H * (P * cached // 2 + 4 * d) + 8), "flops": 4 * c["pages"] * H * P * d}
    mean = (min(c["lo"], c["hi"]) + c["hi"]) / 2
    read = min(mean, c["top_k"] * P) if c["top_k"] else mean
    rows = c["batch"] * H
    return {"bytes": int(rows * read * cached + rows * 4 * (read / P) + c["batch"] * c["hq"] * (d * es + 4 * d + 4)),
            "flops": int(4 * d * read * c["batch"] * c["hq"])}


# ----------------------------------------------- the definitions, in 64 bits --
def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, st)


def _exact_tables(c, st):
    P, B = c["page"], c["batch"]
    a = {k: v.cpu().numpy().astype(np.int64) for k, v in st.items() if isinstance(v, torch.Tensor) and k != "workspace"}
    table, free = a["page_table"], a["free_pages"].tolist()
    slots, pos, ids, valid, lens, cu = [], [], [], [], [], [0]
    taken = refused = 0
    for b in range(B):
        old, new = int(a["seq_lens"][b]), int(a["new_lens"][b])
        cu.append(cu[-1] + new)
        for t in range(old, old + new):
            if t % P == 0:
                table[b, t // P] = free[taken]
                taken += 1
            if t == old or t % P == 0:
                ids.append(table[b, t // P])
                valid.append(min(P, old + new - t // P * P))
            slots.append(table[b, t // P] * P + t % P)
            pos.append(t)
        lens.append(old + new)
    pad = lambda v, like, x: np.concatenate([np.array(v, np.int64), np.full(like.size - len(v), x)])  # noqa: E731
    return dict(page_table=table, seq_lens_out=np.array(lens), cu_new=np.array(cu),
                slot_map=pad(slots, a["slot_map"], -1), positions=pad(pos, a["positions"], -1),
                touched_ids=pad(ids, a["touched_ids"], -1), touched_valid=pad(valid, a["touched_valid"], 0),
                counts=np.array([cu[-1], taken, len(ids), refused]))


def _exact_block(c, raw):
    """Bytes of blocks [..., block bytes] -> keys and values, doubles [..., P, d], by the byte."""
    d, P, NG, gs = c["d"], c["page"], c["d"] // c["gs"], c["gs"]
    dims = torch.arange(d, device=raw.device)
    w, k = dims // 8, dims % 8
    out = []
    t = torch.arange(P, device=raw.device)[:, None]
    for which in (0, 1):
        if which:
            sw = (t // 2) % 4 if d == 128 else (t // 4) % 2
            place = 4 * ((w // 4) ^ sw) + w % 4
        else:
            place = ((w % 4) * (d // 32) + w // 4).expand(P, d)
        byte = raw[..., which * P * d // 2 + t * (d // 2) + 4 * place + k // 2]
        u = torch.where(k % 2 == 1, byte // 16, byte % 16).double()
        par = raw[..., P * d + which * 4 * NG * P:P * d + (which + 1) * 4 * NG * P].contiguous()
        par = par.view(torch.bfloat16).double().unflatten(-1, (NG, P, 2)).transpose(-3, -2)  # [..., P, NG, 2]
        out.append(par[..., 1].repeat_interleave(gs, -1) + par[..., 0].repeat_interleave(gs, -1) * u)
    return out


def _exact_quantised(x, gs):
    """The value that each x stands for once stored."""
    g = x.double().unflatten(-1, (-1, gs))
    m = g.amin(-1, keepdim=True).float().to(torch.bfloat16).double()
    step = (g.amax(-1, keepdim=True) - m).clamp_min(0) / 15
    # one rounding to 8 significant bits
    e = torch.floor(torch.log2(step.clamp_min(2.0 ** -110)))
    e = torch.where(torch.exp2(e) > step, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= step, e + 1, e)
    s = torch.round(step * torch.exp2(7 - e)) * torch.exp2(e - 7)
    s = torch.where(step >= 2.0 ** -100, s, torch.zeros_like(s))
    u = torch.round((g - m) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15)
    return (m + s * u).flatten(-2)


def _exact_append(c, st):
    ok = (st["slots"] >= 0)[:, None, None]
    out = {}
    for n in "kv":
        x = _exact_quantised(st[n], c["gs"])
        out[n] = torch.where(ok, x, torch.zeros_like(x)).cpu()
    return out


def _exact_gather(c, st):
    P, slots = c["page"], st["slots"].long()
    raw = st["pool"]
    out = {"k": [], "v": []}
    step = max(1, (1 << 22) // (P * c["hkv"] * c["d"]))
    for a in range(0, len(slots), step):
        s = slots[a:a + step]
        k, v = _exact_block(c, raw[s.clamp_min(0) // P])  # [n][Hkv][P][d]
        at = (s.clamp_min(0) % P)[:, None, None, None].expand(-1, c["hkv"], 1, c["d"])
        for name, x in (("k", k), ("v", v)):
            x = x.gather(2, at)[:, :, 0]
            out[name].append(torch.where((s >= 0)[:, None, None], x, torch.zeros_like(x)).cpu())
    return {n: torch.cat(x) for n, x in out.items()}


def _exact_meta(c, st):
    meta = torch.zeros(st["meta"].shape, dtype=torch.float64)
    step = max(1, (1 << 24) // (c["page"] * c["hkv"] * c["d"]))
    for a in range(0, c["pages"], step):
        ids = st["page_ids"][a:a + step].long()
        k = _exact_block(c, st["pool"][ids])[0]
        off = (torch.arange(c["page"], device="cuda") >= st["valid"][a:a + step, None])[:, None, :, None]
        lo, hi = k.masked_fill(off, math.inf).amin(2), k.masked_fill(off, -math.inf).amax(2)
        both = []
        for x, to in ((lo, torch.floor), (hi, torch.ceil)):  # outwards, to 8 significant bits
            mag = x.abs().clamp_min(2.0 ** -120)
            e = torch.floor(torch.log2(mag))
            e = torch.where(torch.exp2(e) > mag, e - 1, e)
            e = torch.where(torch.exp2(e + 1) <= mag, e + 1, e)
            both.append(to(x.float().double() * torch.exp2(7 - e)) * torch.exp2(e - 7))
        meta[ids.cpu()] = torch.stack(both, 2).cpu()
    return {"meta": meta}


def _exact_decode(c, st):
    B, H, d, P = c["batch"], c["hkv"], c["d"], c["page"]
    G = c["hq"] // H
    out = torch.zeros((B, H, G, d), dtype=torch.float64)
    lse = torch.full((B, H, G), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(st["seq_lens"][b])
        if n == 0:
            continue
        q = st["q"][b].double().view(H, G, d)
        for h in range(H):
            if c["top_k"]:
                j = st["selected"][b, h, :int(st["n_selected"][b, h])].long()
            else:
                j = torch.arange(-(-n // P), device="cuda")
            if len(j) == 0:
                continue
            k, v = _exact_block(c, st["pool"][st["page_table"][b, j].long(), h])
            on = ((j[:, None] * P + torch.arange(P, device="cuda")) < n).flatten()
            k, v = k.flatten(0, 1)[on], v.flatten(0, 1)[on]
            x = q[h] @ k.T / math.sqrt(d)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            out[b, h] = (p @ v / p.sum(-1, keepdim=True)).cpu()
            lse[b, h] = (top + torch.log(p.sum(-1, keepdim=True)))[:, 0].cpu()
    return {"out": out.view(B, c["hq"], d), "lse": lse.view(B, c["hq"])}
