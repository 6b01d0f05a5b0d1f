"""The paged latent cache: what its three operators compute, over what sizes, and at what cost.

* ``tables``: block tables, slot maps and positions of a step from the requests' lengths;
* ``append``: RMSNorm of the new tokens' latent and RoPE of their key band, written to the
  tokens' slots of the paged cache;
* ``decode``: one query token per request over the paged cache, absorbed MLA form.

``run`` computes them from elementary torch operations, or, where ``own`` is true, through
the library.
"""
import math
import random

import torch

own = False

ROPE_BASE, EPS = 10000.0, 1e-6
DEEPSEEK = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)


def listed():
    return [
        # one serving step: 64 requests at up to 32768 tokens each grow by one token
        dict(name="tables_step_b64", op="tables", batch=64, page=64, past=32768, new=1, spread="ragged"),
        # admission of eight prompts of up to 16384 tokens
        dict(name="tables_prompts_b8", op="tables", batch=8, page=16, past=0, new=16384, spread="ragged"),
        # a large mixed step: decodes and prompt chunks of about two thousand requests
        dict(name="tables_mixed_b2001", op="tables", batch=2001, page=32, past=4096, new=511, spread="ragged"),
        # the cache write of one decode step
        dict(name="append_step_t64", op="append", dtype="bf16", tokens=64, page=64, pages=1024, **DEEPSEEK),
        # the cache write of a 16384-token prompt, latent and key band as views of one projection
        dict(name="append_prompt_t16384", op="append", dtype="bf16", tokens=16384, page=64, pages=1024, **DEEPSEEK),
        # fp32 at small dimensions, an odd page and odd counts
        dict(name="append_fp32_t1001", op="append", dtype="f32", tokens=1001, page=7, pages=160, **TINY),
        # latency: one request of 4096 tokens
        dict(name="decode_b1_l4096_h128", op="decode", dtype="bf16", batch=1, length=4096, heads=128, page=64,
             spread="full", **DEEPSEEK),
        # few long requests
        dict(name="decode_b8_l32768_h128", op="decode", dtype="bf16", batch=8, length=32768, heads=128, page=64,
             spread="full", **DEEPSEEK),
        # the serving batch of the long-context decode, every request at its own length
        dict(name="decode_b64_l32768_h128", op="decode", dtype="bf16", batch=64, length=32768, heads=128, page=64,
             spread="ragged", **DEEPSEEK),
        # the 16-head model: a wide ragged batch over small pages, some requests empty
        dict(name="decode_b200_l4096_h16", op="decode", dtype="bf16", batch=200, length=4096, heads=16, page=16,
             spread="holes", **DEEPSEEK),
        # fp32 at the same dimensions
        dict(name="decode_fp32_b4_l1000_h16", op="decode", dtype="f32", batch=4, length=1000, heads=16, page=32,
             spread="ragged", **DEEPSEEK),
        # fp32 at small dimensions, odd pages
        dict(name="decode_fp32_tiny", op="decode", dtype="f32", batch=5, length=300, heads=4, page=7,
             spread="ragged", **TINY),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "decode", "decode", "decode"])
    if op == "tables":
        batch = _log(rng, 1, 2000)
        new = _log(rng, 1, max(1, min(16384, 500000 // batch)))
        return dict(op=op, batch=batch, page=rng.choice([7, 16, 32, 64, 128]), past=rng.choice([0, _log(rng, 1, 32768)]),
                    new=new, spread=rng.choice(["full", "ragged", "holes"]))
    if op == "append":
        tokens = _log(rng, 1, 16000)
        page = rng.choice([7, 16, 32, 64, 128])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=tokens, page=page,
                    pages=-(-tokens // page) + rng.randint(1, 40), **rng.choice([DEEPSEEK, DEEPSEEK, TINY]))
    dtype, dims = rng.choice([("bf16", DEEPSEEK), ("bf16", DEEPSEEK), ("bf16", DEEPSEEK), ("f32", DEEPSEEK),
                              ("f32", TINY), ("bf16", TINY)])
    small = dtype == "f32" or dims is TINY
    batch = _log(rng, 1, 16 if small else 128)
    return dict(op=op, dtype=dtype, batch=batch, length=_log(rng, 1, 3000 if small else min(32768, 1500000 // batch)),
                heads=rng.choice([1, 4, 8, 16]) if small else rng.choice([8, 16, 20, 32, 64, 128, 128]),
                page=rng.choice([7, 16, 48]) if small else rng.choice([8, 16, 32, 64, 64, 128]),
                spread=rng.choice(["full", "ragged", "holes"]), **dims)


def _lengths(case, count, most, salt):
    """The requests' lengths: a function of the case alone.  full: all `most`; ragged:
    anywhere in [most / 8, most]; holes: the same with every fifth request empty."""
    if case["spread"] == "full" or most == 0:
        return [most] * count
    r = random.Random(1000003 * salt + 31 * count + most)
    got = [r.randint(max(1, most // 8), most) for _ in range(count)]
    if case["spread"] == "holes":
        got = [0 if i % 5 == 2 else n for i, n in enumerate(got)]
    return got


def _tables_lengths(case):
    return _lengths(case, case["batch"], case["past"], 1), _lengths(case, case["batch"], case["new"], 2)


def _pages(n, page):
    return -(-n // page)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1 + seed)

    def normal(*shape, scale=1.0, dtype=None):
        t = torch.randn(*shape, generator=g, device=dev, dtype=dtype or _dtype(case))
        return t if scale == 1.0 else t * scale

    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case)
    if case["op"] == "tables":
        past, new = _tables_lengths(case)
        page = case["page"]
        most = max(_pages(p + n, page) for p, n in zip(past, new)) + 2
        held = [_pages(p, page) for p in past]
        total = sum(_pages(p + n, page) for p, n in zip(past, new))
        ids = torch.randperm(total + 64, generator=g, device=dev).to(torch.int32)
        table = torch.full((case["batch"], most), -1, **i32)
        rows = torch.repeat_interleave(torch.arange(case["batch"], device=dev), torch.tensor(held, device=dev))
        start = torch.tensor([0] + held, device=dev).cumsum(0)
        cols = torch.arange(sum(held), device=dev) - start[rows]
        table[rows, cols] = ids[:sum(held)]
        n = sum(new) + 3   # a padded step: the last rows belong to no request
        s.update(past=torch.tensor(past, **i32), new=torch.tensor(new, **i32), free=ids[sum(held):].contiguous(),
                 table=table, n_tokens=n, kv_lens=torch.empty(case["batch"], **i32),
                 cu=torch.empty(case["batch"] + 1, **i32), slots=torch.empty(n, **i32),
                 positions=torch.empty(n, **i32), counts=torch.empty(2, **i32))
        return s
    if case["op"] == "append":
        n, page, pages = case["tokens"], case["page"], case["pages"]
        kv = normal(n, case["d_kv"] + case["d_rope"])   # one projection gives both
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(n, device=dev)
        slots = order[at // page] * page + at % page
        s.update(kv=kv, c_kv=kv[:, :case["d_kv"]], k_pe=kv[:, case["d_kv"]:],
                 rms_w=(1 + normal(case["d_kv"], scale=0.1)), slots=slots.to(torch.int32),
                 positions=(at + 131 * (seed % 7)).to(torch.int32),
                 c_cache=normal(pages, page, case["d_kv"]), kpe_cache=normal(pages, page, case["d_rope"]))
    else:
        lens = _lengths(case, case["batch"], case["length"], 3)
        page, heads = case["page"], case["heads"]
        per = [_pages(n, page) for n in lens]
        pages = sum(per) + 5
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        most = _pages(case["length"], page) + 1
        table = torch.full((case["batch"], most), -1, **i32)
        rows = torch.repeat_interleave(torch.arange(case["batch"], device=dev), torch.tensor(per, device=dev))
        start = torch.tensor([0] + per, device=dev).cumsum(0)
        table[rows, torch.arange(sum(per), device=dev) - start[rows]] = ids[:sum(per)]
        w = normal(heads * (case["d_nope"] + case["d_v"]), case["d_kv"], scale=1.0 / math.sqrt(case["d_kv"]))
        s.update(q_nope=normal(case["batch"], heads, case["d_nope"]), q_pe=normal(case["batch"], heads, case["d_rope"]),
                 c_cache=normal(pages, page, case["d_kv"]), kpe_cache=normal(pages, page, case["d_rope"]),
                 table=table, kv_lens=torch.tensor(lens, **i32), w=w)
        s["out"] = torch.empty(case["batch"], heads, case["d_v"], dtype=_dtype(case), device=dev)
        s["lse"] = torch.empty(case["batch"], heads, dtype=torch.float32, device=dev)
    if own:
        from head_latent_attention_rmsnorm_gb300 import mla
        s["dims"] = mla.dims(case.get("heads", 1), case["d_kv"], case["d_nope"], case["d_rope"], case["d_v"], ROPE_BASE, EPS)
        if case["op"] == "decode":
            s["workspace"] = mla.paged_decode_workspace(s["dims"], s["c_cache"], s["table"])
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode}[s["op"]](s)


def _run_own(s):
    from head_latent_attention_rmsnorm_gb300 import mla
    if s["op"] == "tables":
        t = mla.paged_tables(s["past"], s["new"], s["free"], s["table"], page_size=s["page"], kv_lens=s["kv_lens"],
                             cu_tokens=s["cu"], slots=s["slots"], positions=s["positions"], counts=s["counts"])
        return dict(table=s["table"], kv_lens=t.kv_lens, cu=t.cu_tokens, slots=t.slots, positions=t.positions, counts=t.counts)
    if s["op"] == "append":
        c, k = mla.paged_append(s["dims"], s["c_kv"], s["k_pe"], s["rms_w"], s["slots"], s["positions"], s["c_cache"],
                                s["kpe_cache"])
        return dict(c_cache=c, kpe_cache=k)
    out, lse = mla.paged_decode(s["dims"], s["q_nope"], s["q_pe"], s["c_cache"], s["kpe_cache"], s["table"], s["kv_lens"],
                                s["w"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ plain forms ----
def _plain_tables(s):
    page, table, n_tokens = s["page"], s["table"], s["n_tokens"]
    past, new, free = s["past"].long(), s["new"].long(), s["free"].long()
    batch, most = table.shape
    cap = most * page
    past = past.clamp(0, cap)
    zero = past.new_zeros(1)
    cu = torch.cat([zero, new.clamp(min=0).cumsum(0)])
    placed = torch.minimum(torch.minimum(new, n_tokens - cu[:-1]), cap - past).clamp(min=0)
    have = (past + page - 1) // page
    extra = (past + placed + page - 1) // page - have
    off = torch.cat([zero, extra.cumsum(0)])
    got = torch.minimum((free.numel() - off[:-1]).clamp(min=0), extra)
    kv = torch.where(got == extra, past + placed, torch.maximum(past, (have + got) * page))
    col = torch.arange(most, device=table.device)
    j = col[None, :] - have[:, None]
    mine = (j >= 0) & (j < got[:, None])
    ids = free[(off[:-1, None] + j).clamp(0, max(free.numel() - 1, 0))] if free.numel() else torch.zeros_like(j)
    table.copy_(torch.where(mine, ids, table.long()))
    t = torch.arange(n_tokens, device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    real = t < cu[-1]
    b = b.clamp(0, batch - 1)
    p = past[b] + t - cu[b]
    ok = real & (p < kv[b])
    slot = torch.where(ok, table[b, (p // page).clamp(0, most - 1)].long() * page + p % page, -1)
    counts = torch.stack([got.sum(), extra.sum()])
    i = torch.int32
    return dict(table=table, kv_lens=kv.to(i), cu=cu.to(i), slots=slot.to(i),
                positions=torch.where(real, p, 0).to(i), counts=counts.to(i))


def _turn(x, pos):
    """RoPE of x [n, ..., d] at positions pos [n]: the angles in 64 bits, the rotation in 32."""
    half = x.shape[-1] // 2
    inv = ROPE_BASE ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / x.shape[-1])
    a = pos.double().reshape([-1] + [1] * (x.dim() - 1)) * inv
    c, n = a.cos().float(), a.sin().float()
    x1, x2 = x[..., :half].float(), x[..., half:].float()
    return torch.cat([x1 * c - x2 * n, x2 * c + x1 * n], -1)


def _plain_append(s):
    x = s["c_kv"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["rms_w"].float()
    at = s["slots"].long()
    c, k = s["c_cache"], s["kpe_cache"]
    c.view(-1, c.shape[-1])[at] = y.to(c.dtype)
    k.view(-1, k.shape[-1])[at] = _turn(s["k_pe"], s["positions"]).to(k.dtype)
    return dict(c_cache=c, kpe_cache=k)


def _plain_decode(s):
    heads, dn, dv, dk = s["heads"], s["d_nope"], s["d_v"], s["d_kv"]
    w = s["w"].float().view(heads, dn + dv, dk)
    lens = s["kv_lens"].long()
    q = torch.einsum("bhn,hnk->bhk", s["q_nope"].float(), w[:, :dn])
    qr = _turn(s["q_pe"], lens - 1)
    table = s["table"].long().clamp(min=0)
    batch, most = table.shape
    seen = torch.arange(most * s["page"], device=table.device)[None] < lens[:, None]
    k = s["c_cache"][table].view(batch, -1, dk).float().masked_fill_(~seen[..., None], 0.0)
    kr = s["kpe_cache"][table].view(batch, -1, s["d_rope"]).float().masked_fill_(~seen[..., None], 0.0)
    scores = torch.matmul(q, k.transpose(1, 2))
    scores += torch.matmul(qr, kr.transpose(1, 2))
    scores *= 1.0 / math.sqrt(dn + s["d_rope"])
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    scores = scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    lse = (total.log() + top)[..., 0].masked_fill(lens[:, None] == 0, -math.inf)
    o = torch.matmul(scores, k) / total.clamp(min=1e-30)
    out = torch.einsum("bhk,hvk->bhv", o, w[:, dn:])
    return dict(out=out.to(s["q_nope"].dtype), lse=lse)


# ------------------------------------------------------------------------ costs ----
def work(case):
    if case["op"] == "tables":
        past, new = _tables_lengths(case)
        taken = sum(_pages(p + n, case["page"]) - _pages(p, case["page"]) for p, n in zip(past, new))
        begun = sum(1 for p, n in zip(past, new) if n and p % case["page"])
        b = case["batch"]
        # lengths in; free pages and partly filled pages' ids in; table entries, lengths, offsets,
        # slots and positions out
        return dict(bytes=4.0 * (2 * b + taken + begun + taken + b + b + 1 + 2 * (sum(new) + 3) + 2), flops=0.0)
    e = 4 if case["dtype"] == "f32" else 2
    width = case["d_kv"] + case["d_rope"]
    if case["op"] == "append":
        n = case["tokens"]
        return dict(bytes=float(n * (2 * width * e + 8) + case["d_kv"] * e), flops=float(n * (4 * case["d_kv"] + 3 * case["d_rope"])))
    lens, h, b = _lengths(case, case["batch"], case["length"], 3), case["heads"], case["batch"]
    keys = sum(lens)
    dn, dv, dk, dr = case["d_nope"], case["d_v"], case["d_kv"], case["d_rope"]
    moved = keys * width * e + h * (dn + dv) * dk * e + b * h * (dn + dr + dv) * e + b * h * 4 + 4 * b
    moved += 4 * sum(_pages(n, case["page"]) for n in lens)
    return dict(bytes=float(moved), flops=float(keys * h * 2 * (2 * dk + dr) + b * h * 2 * dk * (dn + dv)))


# ------------------------------------------------- the definitions, in 64 bits ----
def exact(case, seed):
    if case["op"] == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    f64 = torch.float64
    dev = s["c_cache"].device

    def rotate(x, pos):
        d = x.shape[-1]
        z = torch.complex(x[..., :d // 2].to(f64), x[..., d // 2:].to(f64))
        t = torch.arange(0, d, 2, device=dev, dtype=f64) / d
        ang = pos.to(f64)[:, None] * torch.exp(-t * math.log(ROPE_BASE))
        while ang.dim() < z.dim():
            ang = ang[:, None]
        z = z * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)

    if case["op"] == "append":
        c = s["c_cache"].to(f64).flatten(0, 1)
        k = s["kpe_cache"].to(f64).flatten(0, 1)
        x = s["c_kv"].to(f64)
        where = s["slots"].to(torch.int64)
        c[where] = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * s["rms_w"].to(f64)
        k[where] = rotate(s["k_pe"], s["positions"])
        return dict(c_cache=c.view(s["c_cache"].shape), kpe_cache=k.view(s["kpe_cache"].shape))
    h, dn, dv, dk, dr = case["heads"], case["d_nope"], case["d_v"], case["d_kv"], case["d_rope"]
    w = s["w"].to(f64).view(h, dn + dv, dk)
    wk, wv = w[:, :dn], w[:, dn:]
    lens = s["kv_lens"].tolist()
    out = torch.zeros(case["batch"], h, dv, dtype=f64, device=dev)
    lse = torch.full((case["batch"], h), -math.inf, dtype=f64, device=dev)
    qr = rotate(s["q_pe"], s["kv_lens"].to(f64) - 1)
    for b, n in enumerate(lens):   # request by request
        if n == 0:
            continue
        pages = s["table"][b, :_pages(n, case["page"])].to(torch.int64)
        c = s["c_cache"].index_select(0, pages).flatten(0, 1)[:n].to(f64)
        r = s["kpe_cache"].index_select(0, pages).flatten(0, 1)[:n].to(f64)
        q = torch.matmul(s["q_nope"][b].to(f64)[:, None, :], wk)[:, 0]
        x = (q @ c.T + qr[b] @ r.T) / math.sqrt(dn + dr)
        lse[b] = torch.logsumexp(x, -1)
        out[b] = torch.matmul(wv, (torch.softmax(x, -1) @ c)[:, :, None])[:, :, 0]
    return dict(out=out, lse=lse)
