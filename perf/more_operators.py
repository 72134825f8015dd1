"""Cases of the 8-bit paged KV cache and of prompt attention: what is timed, and their plain forms.

Operators (Hq query heads, Hkv KV heads, G = Hq / Hkv, d = head_dim, P = page_size):

  store    qskv.kvf_append, kvf_gather   new tokens' keys and values stored in 8 bits by slot, and read back as values
  gather   qskv.kvf_gather               cached tokens read back by slot
  meta     qskv.kvf_meta_build           element-wise min / max of a page's cached keys, for the page selection
  decode   qskv.kvf_paged_decode         attention of one query token a sequence over its cached pages, all or a selection
  prefill  qskv.paged_prefill,           causal attention of every sequence's newest tokens, packed one sequence after
           qskv.kvf_paged_prefill        the other, over all that its pages hold (the new tokens among it)

Numbers held in 8 bits.  The d dims x of one token and head (its key, or its value) are stored as
    e = the smallest whole number with max |x| <= 448 * 2^e, clamped to [-100, 119] (-100 where all are zero)
    u = e4m3(x * 2^-e)     (to nearest, ties to even)
and stand for u * 2^e, which bf16 and fp32 hold exactly.

One (page, head) block of the pool is P / 16 parts of 16 tokens each, in bytes:
    [16][d] key codes | [8][d][2] value codes | [16] key e + 127 | [16] value e + 127
16-byte chunk c of a key's row t is stored at place c ^ 4 (t % 2) for d = 128, c for d = 64.  A value row holds two
tokens, dim by dim; its 16-byte chunk c (8 dims) of token pair p is at place c ^ f, f = (p & 1) + 2 (p & 2) for d = 128
and f = 2 (p % 4) for d = 64.

Prefill.  Row b holds seq_lens[b] tokens, of which its last new[b] = cu_new[b + 1] - cu_new[b] are the queries
cu_new[b] .. cu_new[b + 1] of q [T][Hq][d].  Query i of the row stands at pos = seq_lens[b] - new[b] + i and attends to
the tokens 0 .. pos.  Rows of q behind cu_new[batch] are padding: their outputs stay as they were.
"""
import math

import torch

own = False


def _qskv():
    import query_aware_sparse_kv_gb300 as qskv

    return qskv


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a decode step's tokens, one a sequence, from the fused projection's output
        dict(name="store_decode_32", op="store", tokens=32, hq=32, hkv=8, d=128, page=16, dtype="bf16", kind="decode"),
        # a prompt chunk's tokens
        dict(name="store_prompt_32k", op="store", tokens=32_768, hq=32, hkv=8, d=128, page=16, dtype="bf16",
             kind="prefill"),
        # the pages that a decode batch appends to
        dict(name="meta_last_pages_32", op="meta", pages=32, pool=2048, hkv=8, d=128, page=16),
        # every page of a batch after its prompts
        dict(name="meta_prompts_36864", op="meta", pages=36_864, pool=36_900, hkv=8, d=128, page=16),
        # the smallest decode: two short sequences, where latency counts
        dict(name="decode_tiny_fp32", op="decode", batch=2, hq=4, hkv=2, d=64, page=16, lo=1, hi=256, top_k=0,
             dtype="fp32"),
        # the headline batch: 128 selected pages of 4K..32K tokens
        dict(name="decode_gqa4_top128", op="decode", batch=32, hq=32, hkv=8, d=128, page=16, lo=4096, hi=32_768,
             top_k=128, dtype="bf16"),
        # long contexts, all pages, 8 query heads a KV head
        dict(name="decode_long_dense", op="decode", batch=4, hq=64, hkv=8, d=128, page=32, lo=65_536, hi=131_072,
             top_k=0, dtype="bf16"),
        # a few drafted tokens a row checked at once: short, where latency counts
        dict(name="prefill_few_tokens", op="prefill", cache="bf16", batch=4, hq=32, hkv=8, d=128, page=16, new_lo=1,
             new_hi=8, old_lo=0, old_hi=256, kind="prompts", dtype="bf16"),
        # prompts of mixed length, packed
        dict(name="prefill_packed_prompts", op="prefill", cache="bf16", batch=16, hq=32, hkv=8, d=128, page=16,
             new_lo=1, new_hi=4096, old_lo=0, old_hi=0, kind="prompts", dtype="bf16"),
        # one long prompt
        dict(name="prefill_long_prompt", op="prefill", cache="bf16", batch=1, hq=32, hkv=8, d=128, page=16,
             new_lo=16_384, new_hi=16_384, old_lo=0, old_hi=0, kind="prompts", dtype="bf16"),
        # prompts in chunks, over an 8-bit cache of what came before
        dict(name="prefill_chunk_kvf", op="prefill", cache="kvf", batch=4, hq=32, hkv=8, d=128, page=32, new_lo=1024,
             new_hi=2048, old_lo=0, old_hi=30_000, kind="prompts", dtype="bf16"),
        # a small model's prompts in fp32, no shared heads
        dict(name="prefill_mha_fp32", op="prefill", cache="fp32", batch=6, hq=16, hkv=16, d=64, page=16, new_lo=1,
             new_hi=500, old_lo=0, old_hi=77, kind="prompts", dtype="fp32"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["store", "gather", "meta", "decode", "decode", "prefill", "prefill", "prefill"])
    page, d = rng.choice([16, 32]), rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "store":
        kind = rng.choice(["decode", "prefill"])
        tokens = _log(rng, 1, 600) if kind == "decode" else _log(rng, 17, 262_144 // hkv)
        return dict(op=op, tokens=tokens, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=d, page=page,
                    dtype=rng.choice(["bf16", "fp32"]), kind=kind)
    if op == "gather":
        return dict(op=op, tokens=_log(rng, 1, 600_000 // hkv), hkv=hkv, d=d, page=page,
                    dtype=rng.choice(["bf16", "fp32"]))
    if op == "meta":
        pages = _log(rng, 1, 290_000 // hkv // (page // 16))
        return dict(op=op, pages=pages, pool=pages + rng.randrange(1, 100), hkv=hkv, d=d, page=page)
    group = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "decode":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, min(131_072, max(1, 2_000_000 // (batch * hkv))))
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page, lo=rng.choice([0, 1, hi // 2]), hi=hi,
                    top_k=rng.choice([0, 0, 1, 7, 32, 128]), dtype=dtype)
    cache = rng.choice(["bf16", "bf16", "kvf"]) if dtype == "bf16" else rng.choice(["fp32", "bf16", "kvf"])
    batch = _log(rng, 1, 64)
    # (query, token) pairs, all heads, that the padded batch has
    most = (3_000_000_000 if dtype == "bf16" else 400_000_000) // (batch * hkv * group)
    new = _log(rng, 1, min(8192, int(math.sqrt(most))))
    old = rng.choice([0, _log(rng, 1, max(1, min(65_536, most // new - new)))])
    return dict(op=op, cache=cache, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page,
                new_lo=rng.choice([0, 1, new]), new_hi=new, old_lo=rng.choice([0, old // 2, old]), old_hi=old,
                kind=rng.choice(["prompts", "prompts", "mixed"]), dtype=dtype)


# ------------------------------------------------------- the cache's format --
def _block_bytes(c):
    return c["page"] * (2 * c["d"] + 2)


def _part(c, t):
    """First byte of the part that token t of a page lies in."""
    return t // 16 * (16 * (2 * c["d"] + 2))


def _key_places(c, dev):
    """Byte of each dim of a key in its block: [P][d]."""
    t = torch.arange(c["page"], device=dev)[:, None]
    i = torch.arange(c["d"], device=dev)[None, :]
    chunk = i // 16
    if c["d"] == 128:
        chunk = chunk ^ (4 * (t % 2))
    return _part(c, t) + t % 16 * c["d"] + 16 * chunk + i % 16


def _value_places(c, dev):
    """Byte of each dim of a value in its block: [P][d]."""
    t = torch.arange(c["page"], device=dev)[:, None]
    i = torch.arange(c["d"], device=dev)[None, :]
    p = t % 16 // 2
    f = (p & 1) + 2 * (p & 2) if c["d"] == 128 else 2 * (p % 4)
    return _part(c, t) + 16 * c["d"] + p * 2 * c["d"] + 16 * ((i // 8) ^ f) + 2 * (i % 8) + t % 2


def _power_places(c, t, which):
    """Byte of the power of a key (0) or value (1) of token t of a page."""
    return _part(c, t) + 32 * c["d"] + 16 * which + t % 16


def _power(e):
    """2^e of whole e in [-126, 127], as fp32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., d] -> codes uint8 [..., d], e + 127 uint8 [...]."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e, torch.full_like(e, -100)).clamp(-100, 119)
    u = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return u.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, exps):
    """The fp32 numbers that codes [..., d] with e + 127 [...] stand for."""
    return codes.view(torch.float8_e4m3fn).float() * _power(exps.to(torch.int32) - 127)[..., None]


def _store(c, pool, slots, k, v):
    """Tokens k, v [n][Hkv][d] into the slots of pool [Npool][Hkv][block bytes]."""
    P, H = c["page"], c["hkv"]
    # a negative slot repeats the first token's store
    keep = torch.where(slots >= 0, torch.arange(len(slots), device=slots.device), 0)
    slot = slots[keep].long()
    t = slot % P
    base = ((slot // P * H)[:, None] + torch.arange(H, device=slot.device)) * _block_bytes(c)
    flat = pool.view(-1)
    for which, (x, places) in enumerate(((k, _key_places), (v, _value_places))):
        codes, exps = _quantise(x[keep])
        flat[base[:, :, None] + places(c, slot.device)[t][:, None, :]] = codes
        flat[base + _power_places(c, t, which)[:, None]] = exps


def _read(c, pool, slots, which, dtype):
    """Values [n][Hkv][d] of the slots (0 where a slot is negative)."""
    P, H = c["page"], c["hkv"]
    slot = slots.clamp_min(0).long()
    t = slot % P
    base = ((slot // P * H)[:, None] + torch.arange(H, device=slot.device)) * _block_bytes(c)
    places = (_value_places if which else _key_places)(c, slot.device)
    flat = pool.view(-1)
    x = _values(flat[base[:, :, None] + places[t][:, None, :]], flat[base + _power_places(c, t, which)[:, None]])
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(dtype)


def _unpack(c, blocks, which):
    """Blocks [..., block bytes] -> values fp32 [..., P, d] of the keys (0) or the values (1)."""
    codes = blocks[..., (_value_places if which else _key_places)(c, blocks.device)]
    return _values(codes, blocks[..., _power_places(c, torch.arange(c["page"], device=blocks.device), which)])


# ------------------------------------------------------------------ inputs --
def _dtype(c):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[c["dtype"]]


def _keys(g, *shape):
    """Keys or values as projections make them: some dims with an offset and a larger spread."""
    d = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda")
    spread = 0.5 + torch.rand(d, generator=g, device="cuda")
    return x * spread + 2.0 * torch.randn(d, generator=g, device="cuda") * (torch.rand(d, generator=g, device="cuda") < 0.1)


def _pool8(c, g, pages):
    """A pool of `pages` pages of keys and values in 8 bits."""
    d, P, H = c["d"], c["page"], c["hkv"]
    pool = torch.empty((pages, H, _block_bytes(c)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (P * H * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for which in (0, 1):
            codes, exps = _quantise(_keys(g, n, H, P, d))
            pool[a:a + n, :, (_value_places if which else _key_places)(c, pool.device).flatten()] = codes.flatten(-2)
            pool[a:a + n, :, _power_places(c, torch.arange(P, device=pool.device), which)] = exps
    return pool


def _pool16(c, g, pages):
    """Keys (or values) [pages][Hkv][P][d] in bf16 or fp32."""
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[c["cache"]]
    pool = torch.empty((pages, c["hkv"], c["page"], c["d"]), dtype=dt, device="cuda")
    step = max(1, (1 << 25) // (c["page"] * c["hkv"] * c["d"]))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        pool[a:a + n] = _keys(g, n, c["hkv"], c["page"], c["d"]).to(dt)
    return pool


def _table(g, lens, P, max_pages):
    """Page table of rows of `lens` tokens over randomly ordered pages, and the pages of the pool."""
    n = (lens + P - 1) // P
    total = int(n.sum())
    ids = torch.randperm(total + 5, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(max_pages, device="cuda")[None, :]
    start = (torch.cumsum(n, 0) - n)[:, None]
    table = torch.where(j < n[:, None], ids[(start + j).clamp(max=total + 4)], torch.full_like(ids[:1], -1))
    return table.contiguous(), total + 5


def _spoil(c, st, lens):
    """Slots past a row's end hold whatever was there before: not numbers."""
    P, d = c["page"], c["d"]
    last = torch.nonzero(lens % P).flatten()
    page = st["page_table"][last, lens[last] // P].long()
    bad = torch.arange(P, device="cuda")[None, :] >= (lens[last] % P)[:, None]  # [rows][P]
    if "pool" in st:
        b = st["pool"][page]
        for which, places in enumerate((_key_places, _value_places)):
            x = places(c, b.device).flatten()
            b[:, :, x] = torch.where(bad[:, None, :, None], 0x7F, b[:, :, x].unflatten(-1, (P, d))).flatten(-2)
            x = _power_places(c, torch.arange(P, device=b.device), which)
            b[:, :, x] = torch.where(bad[:, None, :], 0xFF, b[:, :, x])
        st["pool"][page] = b
    else:
        for n in ("k_pool", "v_pool"):
            st[n][page] = st[n][page].masked_fill(bad[:, None, :, None], math.nan)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    P, H, d = c["page"], c["hkv"], c["d"]
    ints = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] in ("store", "gather"):
        n = c["tokens"]
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
        st["k_out"], st["v_out"] = (torch.empty((n, H, d), dtype=_dtype(c), device="cuda") for _ in range(2))
        if c["op"] == "store":
            qkv = torch.cat([torch.randn((n, c["hq"], d), generator=g, device="cuda"), _keys(g, n, H, d),
                             _keys(g, n, H, d)], 1).to(_dtype(c))
            st["k"], st["v"] = qkv[:, c["hq"]:c["hq"] + H], qkv[:, c["hq"] + H:]
            st["pool"] = torch.zeros((pages, H, _block_bytes(c)), dtype=torch.uint8, device="cuda")
        else:
            st["pool"] = _pool8(c, g, pages)
        shape = (1, c.get("hq", H), H, d, P, 1, pages)
    elif c["op"] == "meta":
        st["pool"] = _pool8(c, g, c["pool"])
        st["page_ids"] = torch.randperm(c["pool"], generator=g, device="cuda")[:c["pages"]].to(torch.int32)
        st["valid"] = torch.where(torch.rand(c["pages"], generator=g, device="cuda") < 0.1, ints(1, P, c["pages"]),
                                  torch.full((c["pages"],), P, device="cuda")).to(torch.int32)
        st["meta"] = torch.zeros((c["pool"], H, 2, d), dtype=torch.bfloat16, device="cuda")
        shape = (1, H, H, d, P, 1, c["pool"])
    elif c["op"] == "decode":
        B = c["batch"]
        lens = ints(min(c["lo"], c["hi"]), c["hi"], B)
        lens[0].clamp_(min=1)  # some row has work
        mp = max(1, -(-c["hi"] // P))
        st["page_table"], pages = _table(g, lens, P, mp)
        st.update(pool=_pool8(c, g, pages), seq_lens=lens.to(torch.int32))
        _spoil(c, st, lens)
        st["q"] = torch.randn((B, c["hq"], d), generator=g, device="cuda").to(_dtype(c))
        st["out"] = torch.empty((B, c["hq"], d), device="cuda")
        st["lse"] = torch.empty((B, c["hq"]), device="cuda")
        if c["top_k"]:
            K, n = c["top_k"], (lens + P - 1) // P
            j = torch.arange(mp, device="cuda")
            key = torch.rand((B, H, mp), generator=g, device="cuda").masked_fill_((j >= n[:, None])[:, None, :], 2.0)
            pick = key.argsort(-1)[..., :K].to(torch.int32)
            past = torch.arange(pick.shape[-1], device="cuda") >= n[:, None, None]
            pick = pick.masked_fill(past, 1 << 30).sort(-1).values
            pick = pick.masked_fill(pick == 1 << 30, -1)
            st["selected"] = torch.nn.functional.pad(pick, (0, K - pick.shape[-1]), value=-1).contiguous()
            st["n_selected"] = n.clamp(max=K).to(torch.int32)[:, None].expand(B, H).contiguous()
        shape = (B, c["hq"], H, d, P, mp, pages)
    else:
        B = c["batch"]
        new, old = ints(c["new_lo"], c["new_hi"], B), ints(c["old_lo"], c["old_hi"], B)
        if c["kind"] == "mixed":  # two rows in three run on by a token
            new = torch.where(torch.rand(B, generator=g, device="cuda") < 2 / 3, torch.ones_like(new), new)
        new[0].clamp_(min=1)
        lens = old + new
        mp = max(1, -(-(c["old_hi"] + max(1, c["new_hi"])) // P))
        st["page_table"], pages = _table(g, lens, P, mp)
        st["seq_lens"] = lens.to(torch.int32)
        st["cu_new"] = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)]).to(torch.int32)
        if c["cache"] == "kvf":
            st["pool"] = _pool8(c, g, pages)
        else:
            st["k_pool"], st["v_pool"] = _pool16(c, g, pages), _pool16(c, g, pages)
        _spoil(c, st, lens)
        T = B * max(1, c["new_hi"]) + 3  # buffers for the longest step: the rows behind cu_new[B] are padding
        # the queries as the fused projection leaves them, a view of its output
        qkv = torch.randn((T, c["hq"] + 2 * H, d), generator=g, device="cuda").to(_dtype(c))
        st["q"] = qkv[:, :c["hq"]]
        st["out"] = torch.zeros((T, c["hq"], d), dtype=_dtype(c), device="cuda")
        st["lse"] = torch.zeros((T, c["hq"]), device="cuda")
        shape = (B, c["hq"], H, d, P, mp, pages)
    if own:
        st["shape"] = _qskv().make_shape(*shape)
        size = 256
        if c["op"] == "decode":
            size = _qskv().kvf_workspace_size(st["shape"])
        elif c["op"] == "prefill":
            size = _qskv().prefill_workspace_size(st["shape"], len(st["q"]))
        st["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------- one pass --
def run(st):
    return globals()["_run_" + st["case"]["op"]](st)


def _run_store(st):
    """Tokens stored, and read back as the values that the cache then stands for."""
    c = st["case"]
    if own:
        _qskv().kvf_append(st["k"], st["v"], st["slots"], st["pool"], st["shape"], st["workspace"])
        _qskv().kvf_gather(st["pool"], st["slots"], st["k_out"], st["v_out"], st["shape"], st["workspace"])
        return {"k": st["k_out"], "v": st["v_out"]}
    _store(c, st["pool"], st["slots"], st["k"], st["v"])
    return _run_gather(st)


def _run_gather(st):
    c = st["case"]
    if own:
        _qskv().kvf_gather(st["pool"], st["slots"], st["k_out"], st["v_out"], st["shape"], st["workspace"])
        return {"k": st["k_out"], "v": st["v_out"]}
    return {"k": _read(c, st["pool"], st["slots"], 0, _dtype(c)), "v": _read(c, st["pool"], st["slots"], 1, _dtype(c))}


def _run_meta(st):
    c = st["case"]
    if own:
        _qskv().kvf_meta_build(st["pool"], st["page_ids"], st["valid"], st["meta"], st["shape"], st["workspace"])
        return {"meta": st["meta"]}
    ids = st["page_ids"].long()
    k = _unpack(c, st["pool"][ids], 0)  # [n][Hkv][P][d]
    off = (torch.arange(c["page"], device=ids.device) >= st["valid"][:, None])[:, None, :, None]
    st["meta"][ids] = torch.stack([k.masked_fill(off, math.inf).amin(2), k.masked_fill(off, -math.inf).amax(2)],
                                  2).to(torch.bfloat16)
    return {"meta": st["meta"]}


def _softmax_times(x, v):
    """Softmax of x (overwritten) over its last axis times v, and log sum exp; 0 and -inf where all of a row is -inf."""
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    return (x @ v) / total.clamp_min(1e-30), (top + torch.log(total))[..., 0]


def _run_decode(st):
    c = st["case"]
    if own:
        _qskv().kvf_paged_decode(st["q"], st["pool"], st["page_table"], st["seq_lens"], st["out"], st["shape"],
                                 st["workspace"], selected=st.get("selected"), n_selected=st.get("n_selected"),
                                 top_k=c["top_k"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    B, H, d, P = c["batch"], c["hkv"], c["d"], c["page"]
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
    blocks = st["pool"][page.clamp_min(0), torch.arange(H, device=table.device)[None, :, None]]
    q = st["q"].float().view(B, H, -1, d)
    x = (q @ _unpack(c, blocks, 0).flatten(2, 3).transpose(-1, -2)) / math.sqrt(d)
    v = _unpack(c, blocks, 1).flatten(2, 3).masked_fill_(off.transpose(-1, -2), 0.0)
    o, lse = _softmax_times(x.masked_fill_(off, -math.inf), v)
    return {"out": o.reshape(B, c["hq"], d), "lse": lse.reshape(B, c["hq"])}


def _run_prefill(st):
    c = st["case"]
    if own:
        if c["cache"] == "kvf":
            _qskv().kvf_paged_prefill(st["q"], st["pool"], st["page_table"], st["seq_lens"], st["cu_new"], st["out"],
                                      st["shape"], st["workspace"], lse=st["lse"])
        else:
            _qskv().paged_prefill(st["q"], st["k_pool"], st["v_pool"], st["page_table"], st["seq_lens"], st["cu_new"],
                                  st["out"], st["shape"], st["workspace"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    B, H, d = c["batch"], c["hkv"], c["d"]
    G, T, dev = c["hq"] // H, len(st["q"]), st["q"].device
    lens, cu, page = st["seq_lens"].long(), st["cu_new"].long(), st["page_table"].long().clamp_min(0)
    N = max(1, c["new_hi"])
    # the batch, padded: [B][H][queries x G][d] over [B][H][tokens][d]
    i = torch.arange(N, device=dev)[None, :]
    at = torch.where(cu[:-1, None] + i < cu[1:, None], cu[:-1, None] + i, T)  # T: none
    q = st["q"][at.clamp(max=T - 1)].float().view(B, N, H, G, d).transpose(1, 2).reshape(B, H, N * G, d)
    pools = (st["pool"],) * 2 if c["cache"] == "kvf" else (st["k_pool"], st["v_pool"])
    k, v = ((_unpack(c, p[page], w) if c["cache"] == "kvf" else p[page].float()).transpose(1, 2).flatten(2, 3)
            for w, p in enumerate(pools))
    t = torch.arange(k.shape[2], device=dev)
    v.masked_fill_((t >= lens[:, None])[:, None, :, None], 0.0)
    x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    pos = (lens - cu[1:] + cu[:-1])[:, None] + i  # [B][N]
    x.view(B, H, N, G, -1).masked_fill_((t > pos[..., None])[:, None, :, None, :], -math.inf)
    o, lse = _softmax_times(x, v)
    o = o.view(B, H, N, G, d).transpose(1, 2).reshape(B, N, c["hq"], d).to(_dtype(c))
    out, sums = (torch.cat([y, torch.zeros_like(y[:1])]) for y in (st["out"], st["lse"]))
    out[at] = o
    sums[at] = lse.view(B, H, N, G).transpose(1, 2).reshape(B, N, c["hq"])
    return {"out": out[:T], "lse": sums[:T]}


# -------------------------------------------------- what a pass cannot avoid --
def _mean(lo, hi):
    return (lo + hi) / 2


def work(case):
    c = case
    P, d, H = c["page"], c["d"], c["hkv"]
    cached = 2 * d + 2  # bytes of one token and head, keys and values
    es = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "store":
        n = c["tokens"]
        return {"bytes": n * H * (2 * d * es + 2 * cached + 2 * d * es) + 8 * n, "flops": 4 * n * H * 2 * d}
    if c["op"] == "gather":
        n = c["tokens"]
        return {"bytes": n * H * (cached + 2 * d * es) + 4 * n, "flops": 2 * n * H * d}
    if c["op"] == "meta":
        return {"bytes": c["pages"] * (H * (P * cached // 2 + 4 * d) + 8), "flops": 3 * c["pages"] * H * P * d}
    if c["op"] == "decode":
        mean = _mean(min(c["lo"], c["hi"]), c["hi"])
        read = min(mean, c["top_k"] * P) if c["top_k"] else mean
        rows = c["batch"] * H
        return {"bytes": int(rows * read * cached + rows * 4 * (read / P) + c["batch"] * c["hq"] * (d * es + 4 * d + 4)),
                "flops": int(4 * d * read * c["batch"] * c["hq"])}
    if c["cache"] != "kvf":
        cached = 2 * d * (2 if c["cache"] == "bf16" else 4)
    # means over the rows' lengths (whole numbers of a range, independent of each other)
    lo, hi, old = c["new_lo"], c["new_hi"], _mean(c["old_lo"], c["old_hi"])
    new, square = _mean(lo, hi), _mean(lo, hi) ** 2 + ((hi - lo + 1) ** 2 - 1) / 12
    if c["kind"] == "mixed":
        new, square = (2 + new) / 3, (2 + square) / 3
    pairs = c["batch"] * (square / 2 + new / 2 + new * old)
    tokens = c["batch"] * new
    return {"bytes": int(c["batch"] * (new + old) * H * (cached + 4 / H / P) + tokens * c["hq"] * (2 * d * es + 4)) + 4,
            "flops": int(4 * d * c["hq"] * pairs)}


# ----------------------------------------------- the definitions, in 64 bits --
def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, st)


def _exact_number(b):
    """The numbers of e4m3 bytes, from their bits."""
    b = b.long()
    e, m = (b >> 3) & 15, b & 7
    x = torch.where(e == 0, m.double() / 512, (8 + m).double() * torch.exp2((e - 10).double()))
    return torch.where(b >= 128, -x, x)


def _exact_block(c, raw):
    """Bytes of blocks [..., block bytes] -> keys and values, doubles [..., P, d], by the byte."""
    P, d = c["page"], c["d"]
    raw = raw.unflatten(-1, (P // 16, 32 * d + 32))  # parts of 16 tokens
    dims, t = torch.arange(d, device=raw.device), torch.arange(16, device=raw.device)[:, None]
    if d == 128:
        key = dims % 16 + ((dims // 16 + 4 * (t % 2)) % 8) * 16
        turn = t // 2 % 2 + 4 * (t // 4 % 2)
    else:
        key, turn = dims.expand(16, d), 2 * (t // 2 % 4)
    value = t // 2 * 2 * d + (dims // 8 ^ turn) * 16 + dims % 8 * 2 + t % 2
    power = torch.exp2(raw[..., 32 * d:].double() - 127)
    k = _exact_number(raw[..., t * d + key]) * power[..., :16, None]
    v = _exact_number(raw[..., 16 * d + value]) * power[..., 16:, None]
    k, v = k.flatten(-3, -2), v.flatten(-3, -2)
    return k, v


def _exact_store(c, st):
    """Each value once stored: rounded to 4 significant bits, or to multiples of 2^(e - 9) where that is coarser."""
    ok = (st["slots"] >= 0)[:, None, None]
    out = {}
    for n in "kv":
        x = st[n].double()
        top = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / 448))
        e = torch.where(448 * torch.exp2(e) < top, e + 1, e)
        e = torch.where(448 * torch.exp2(e - 1) >= top, e - 1, e).clamp(-100, 119)
        y = x * torch.exp2(-e)
        p = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20)))
        p = torch.where(torch.exp2(p) > y.abs(), p - 1, p)
        p = torch.where(torch.exp2(p + 1) <= y.abs(), p + 1, p)
        step = torch.exp2(p.clamp_min(-6) - 3)
        x = torch.round(y / step) * step * torch.exp2(e)
        out[n] = torch.where(ok, x, torch.zeros_like(x))
    return out


def _exact_gather(c, st):
    P, slots = c["page"], st["slots"].long()
    out = {"k": [], "v": []}
    step = max(1, (1 << 22) // (P * c["hkv"] * c["d"]))
    for a in range(0, len(slots), step):
        s = slots[a:a + step]
        at = (s.clamp_min(0) % P)[:, None, None, None].expand(-1, c["hkv"], 1, c["d"])
        for n, x in zip("kv", _exact_block(c, st["pool"][s.clamp_min(0) // P])):
            x = x.gather(2, at)[:, :, 0]
            out[n].append(torch.where((s >= 0)[:, None, None], x, torch.zeros_like(x)))
    return {n: torch.cat(x) for n, x in out.items()}


def _exact_meta(c, st):
    meta = torch.zeros(st["meta"].shape, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 24) // (c["page"] * c["hkv"] * c["d"]))
    for a in range(0, c["pages"], step):
        ids = st["page_ids"][a:a + step].long()
        k = _exact_block(c, st["pool"][ids])[0]
        off = (torch.arange(c["page"], device="cuda") >= st["valid"][a:a + step, None])[:, None, :, None]
        meta[ids] = torch.stack([k.masked_fill(off, math.inf).amin(2), k.masked_fill(off, -math.inf).amax(2)], 2)
    return {"meta": meta}


def _exact_decode(c, st):
    B, H, d, P = c["batch"], c["hkv"], c["d"], c["page"]
    G = c["hq"] // H
    out = torch.zeros((B, H, G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, G), -math.inf, dtype=torch.float64, device="cuda")
    lens = st["seq_lens"].tolist()
    for b in range(B):
        for h in range(H):
            if c["top_k"]:
                j = st["selected"][b, h, :int(st["n_selected"][b, h])].long()
            else:
                j = torch.arange(-(-lens[b] // P), device="cuda")
            if len(j) == 0:
                continue
            k, v = _exact_block(c, st["pool"][st["page_table"][b, j].long(), h])
            on = ((j[:, None] * P + torch.arange(P, device="cuda")) < lens[b]).flatten()
            k, v = k.flatten(0, 1)[on], v.flatten(0, 1)[on]
            x = st["q"][b, h * G:(h + 1) * G].double() @ k.T * d ** -0.5
            lse[b, h] = torch.logsumexp(x, -1)
            out[b, h] = torch.softmax(x, -1) @ v
    return {"out": out.view(B, c["hq"], d), "lse": lse.view(B, c["hq"])}


def _exact_prefill(c, st):
    H, d, P = c["hkv"], c["d"], c["page"]
    G = c["hq"] // H
    out, lse = st["out"].double(), st["lse"].double()
    cu, lens = st["cu_new"].tolist(), st["seq_lens"].tolist()
    for b in range(c["batch"]):
        if cu[b] == cu[b + 1]:
            continue
        pages = st["page_table"][b, :-(-lens[b] // P)].long()
        for h in range(H):
            if c["cache"] == "kvf":
                k, v = _exact_block(c, st["pool"][pages, h])
            else:
                k, v = st["k_pool"][pages, h].double(), st["v_pool"][pages, h].double()
            k, v = k.flatten(0, 1)[:lens[b]], v.flatten(0, 1)[:lens[b]]
            for a in range(cu[b], cu[b + 1], 2048):
                e = min(a + 2048, cu[b + 1])
                first = lens[b] - cu[b + 1] + a  # the position of query a
                n = first + e - a
                q = st["q"][a:e, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,td->gnt", q, k[:n]) * d ** -0.5
                late = torch.arange(n, device="cuda")[None, :] > first + torch.arange(e - a, device="cuda")[:, None]
                x = x.masked_fill(late, -math.inf)
                lse[a:e, h * G:(h + 1) * G] = torch.logsumexp(x, -1).T
                out[a:e, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", torch.softmax(x, -1), v[:n])
    return {"out": out, "lse": lse}
