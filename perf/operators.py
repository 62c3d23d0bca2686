"""The measured operators: sliding-window attention over a latent cache, a latent cache held in
4 bits (attention, append, read-back), and page bookkeeping of a paged cache.

Geometry of the library: 64 heads, a latent of 512, pages of 64 rows, softmax scale 1/16.
"""
import math

import torch

own = False

H, R, PAGE, GROUP = 64, 512, 64, 16
SCALE = 1.0 / 16.0
ROW_BYTES = R // 2 + R // GROUP  # a packed row: 256 bytes of 4-bit codes, then 32 scales


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of 32 sequences that attend their last 4,096 rows and 64 first ones
        dict(name="window_dense_decode", op="window", paged=False, B=32, Q=1, lo=8192, hi=8192, window=4096, sinks=64),
        # a verify step (1 token + 5 drafts) over ragged paged sequences, odd window, a few sinks
        dict(name="window_paged_verify", op="window", paged=True, B=16, Q=6, lo=1024, hi=32774, window=4095, sinks=5),
        # one short conversation: latency
        dict(name="packed_tiny", op="packed", B=1, Q=1, lo=256, hi=256, window=0, sinks=0, unit=1.0),
        # a decode step of 32 sequences of 8,192 rows
        dict(name="packed_decode", op="packed", B=32, Q=1, lo=8192, hi=8192, window=0, sinks=0, unit=1.0),
        # long ragged contexts: what the 4-bit cache is for
        dict(name="packed_ragged", op="packed", B=16, Q=1, lo=1024, hi=131072, window=0, sinks=0, unit=0.125),
        # a verify step with window and sinks over 4-bit rows
        dict(name="packed_window_verify", op="packed", B=16, Q=6, lo=1024, hi=32774, window=8191, sinks=64, unit=1.0),
        # the append of a verify step
        dict(name="append_verify", op="append", B=32, Q=6, lo=1, hi=8192, unit=1.0),
        # the append of prompts
        dict(name="append_prompt", op="append", B=8, Q=4001, lo=0, hi=2048, unit=0.125),
        # a sampling step over a few sequences: two end, two are forked, all get room for a verify window
        dict(name="beam_small", op="beam", B=8, Q=6, lo=100, hi=1000, forks=2, packed=False),
        # the same over a full batch
        dict(name="beam_large", op="beam", B=256, Q=6, lo=1024, hi=4096, forks=96, packed=False),
        # a small pool after some sequences ended
        dict(name="compact_small", op="compact", B=8, lo=100, hi=1000, keep=0.5, packed=True),
        # a pool of a full batch, half of it free
        dict(name="compact_large", op="compact", B=128, lo=1024, hi=8192, keep=0.5, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("window", "packed", "packed", "append", "beam", "compact"))
    if op in ("window", "packed"):
        Q = rng.choice((1, 1, 2, 3, 6, 8))
        B = _log(rng, 1, 32)
        hi = _log(rng, 64, 131072)
        while B * hi > 32 * 8192 or B * Q * hi > 16 * 32774:
            B = max(1, B // 2)
            Q = max(1, Q // 2)
            if B == 1 and Q == 1:
                break
        c = dict(op=op, B=B, Q=Q, lo=max(Q, hi // rng.choice((1, 2, 8))), hi=hi)
        c["window"] = _log(rng, 1, 8192)
        c["sinks"] = rng.choice((0, 1, 4, 63, 64, 200))
        if op == "window":
            c["paged"] = rng.random() < 0.5
        else:
            c["unit"] = rng.choice((1.0, 0.125, 4.0))
            if rng.random() < 0.5:
                c["window"] = c["sinks"] = 0
        return c
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Q=_log(rng, 1, max(2, 32768 // B)), lo=0, hi=_log(rng, 2, 4096), unit=rng.choice((1.0, 0.125, 4.0)))
    B = _log(rng, 4, 128)
    hi = _log(rng, 64, 4096)
    if op == "beam":
        return dict(op=op, B=B, Q=rng.choice((1, 2, 6, 64, 100)), lo=max(1, hi // 4), hi=hi, forks=rng.randint(1, max(1, B // 3)), packed=rng.random() < 0.5)
    return dict(op=op, B=B, lo=max(1, hi // 4), hi=hi, keep=rng.choice((0.25, 0.5, 0.75)), packed=rng.random() < 0.5)


# ----------------------------------------------------------------------------- the packed row
def e2m1_table(dtype, device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=dtype, device=device)


def quantise(x, unit):
    """x [..., 512] float32 -> bytes [..., 288]: one e4m3 scale per 16 values, e2m1 codes."""
    y = (x / unit).unflatten(-1, (R // GROUP, GROUP))
    amax = y.abs().amax(-1, keepdim=True)
    scale = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    q = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = (code + 8 * torch.signbit(q).to(torch.uint8)).flatten(-2)
    return torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1).view(torch.uint8)], dim=-1)


def dequantise(p, unit, dtype=torch.float32):
    """bytes [..., 288] -> values [..., 512]."""
    c = p[..., : R // 2]
    code = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)
    v = e2m1_table(dtype, p.device)[code.int()]
    s = p[..., R // 2 :].contiguous().view(torch.float8_e4m3fn).to(dtype) * unit
    return (v.unflatten(-1, (R // GROUP, GROUP)) * s.unsqueeze(-1)).flatten(-2)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lens(g, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)


def _table(g, pages_of, max_pages, num_pages):
    """A shuffled page table: sequence b maps its first pages_of[b] entries, the others are -1."""
    k = torch.arange(max_pages, device="cuda")
    used = k[None] < pages_of[:, None]
    rank = (used.flatten().long().cumsum(0) - 1).view_as(used)
    perm = torch.randperm(num_pages, generator=g, device="cuda")
    return torch.where(used, perm[rank.clamp(0, num_pages - 1)], -1).to(torch.int32)


def _rows(g, *shape):
    """Latent rows: normal values, channels of unlike spread."""
    gain = torch.exp(0.5 * torch.randn(R, generator=g, device="cuda"))
    return (torch.randn(*shape, R, generator=g, device="cuda") * gain).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op, B = case["op"], case["B"]
    s = dict(case=case)
    if op in ("window", "packed"):
        Q = case["Q"]
        lens = _lens(g, B, case["lo"], case["hi"])
        s["seq_lens"] = lens
        s["qt"] = (torch.randn(B, Q, H, R, generator=g, device="cuda") * math.sqrt(0.5)).to(torch.bfloat16)
        if op == "window" and not case["paged"]:
            s["cache"] = torch.randn(B, case["hi"], R, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        else:
            max_pages = -(-case["hi"] // PAGE)
            num_pages = B * max_pages
            s["page_table"] = _table(g, -(-lens.long() // PAGE), max_pages, num_pages)
            if op == "window":
                s["pool"] = torch.randn(num_pages, PAGE, R, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
            else:
                s["pool"] = torch.empty(num_pages, PAGE, ROW_BYTES, dtype=torch.uint8, device="cuda")
                for a in range(0, num_pages, 4096):
                    part = s["pool"][a : a + 4096]
                    part.copy_(quantise(_rows(g, part.shape[0], PAGE).float() * case["unit"], case["unit"]))
        if own:
            import mla_absorbed_latent_mtp_b200 as m
            s["workspace"] = m.new_workspace(B, Q)
    elif op == "append":
        Q = case["Q"]
        lens = _lens(g, B, case["lo"], case["hi"])
        max_pages = -(-(case["hi"] + Q) // PAGE)
        s["page_table"] = _table(g, -(-(lens.long() + Q) // PAGE), max_pages, B * max_pages)
        s["pool"] = torch.zeros(B * max_pages, PAGE, ROW_BYTES, dtype=torch.uint8, device="cuda")
        s["rows"] = (_rows(g, B, Q).float() * case["unit"]).to(torch.bfloat16)
        s["start"], s["seq_lens"] = lens, lens.clone()
    else:
        lens = _lens(g, B, case["lo"], case["hi"])
        max_pages = -(-(case["hi"] + case.get("Q", 0)) // PAGE) + 1
        num_pages = B * max_pages
        table = _table(g, -(-lens.long() // PAGE), max_pages, num_pages)
        perm = torch.randperm(B, generator=g, device="cuda").to(torch.int32)
        if op == "beam":
            n = case["forks"]
            s["children"], s["parents"] = perm[:n].contiguous(), perm[n : 2 * n].contiguous()
        else:  # some of the sequences have ended and their pages are free
            table[perm[int(B * case["keep"]) :].long()] = -1
        refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        refs.index_add_(0, table.flatten().clamp(min=0).long(), (table.flatten() >= 0).to(torch.int32))
        s["table0"], s["lens0"], s["refs0"] = table, lens, refs
        s["page_table"], s["seq_lens"], s["refs"] = table.clone(), lens.clone(), refs.clone()
        if case["packed"]:
            s["pool"] = torch.randint(0, 256, (num_pages, PAGE, ROW_BYTES), generator=g, device="cuda", dtype=torch.uint8)
        else:
            s["pool"] = torch.randn(num_pages, PAGE, R, generator=g, device="cuda", dtype=torch.bfloat16)
        if own:
            import mla_absorbed_latent_mtp_b200 as m
            s["workspace"] = m.new_pages_workspace(B, num_pages)
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def positions(case, lens, last):
    """Positions [B, n] that a step may look at (the sinks, then the window of the Q queries, or
    every row), and whether each is a row of its own and of the cache."""
    if case["window"] == 0:
        j = torch.arange(last, device=lens.device).expand(lens.numel(), last)
        return j, j < lens[:, None]
    lens = lens.long()
    sinks = torch.arange(min(case["sinks"], last), device=lens.device).expand(lens.numel(), -1)
    n = case["window"] + case["Q"] - 1
    recent = lens[:, None] - n + torch.arange(n, device=lens.device)
    j = torch.cat([sinks, recent], dim=1)
    fine = torch.cat([sinks < lens[:, None], recent >= sinks.shape[1]], dim=1)
    return j.clamp(0, last - 1), fine


def visible(case, lens, j, fine):
    """[B, Q, n]: what each query sees."""
    t = lens.long()[:, None] - case["Q"] + torch.arange(case["Q"], device=lens.device)
    see = fine[:, None, :] & (j[:, None, :] <= t[:, :, None])
    if case["window"]:
        see = see & ((t[:, :, None] - j[:, None, :] < case["window"]) | (j[:, None, :] < case["sinks"]))
    return see


def attend(qt, rows, see):
    """qt [B, Q, H, R], rows [B, n, R], see [B, Q, n] -> o [B, Q, H, R], lse [B, Q, H]."""
    B, Q = qt.shape[:2]
    score = torch.bmm(qt.flatten(1, 2), rows.transpose(1, 2)).view(B, Q, H, -1) * SCALE
    score = score.masked_fill(~see[:, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp(min=1e-30)
    o = torch.bmm(p.flatten(1, 2), rows).view(B, Q, H, R)
    return o, (top + torch.log(total)).squeeze(-1)


def gather(s, j):
    """Stored rows at positions j [B, n] of each sequence."""
    b = torch.arange(j.shape[0], device=j.device)[:, None]
    if "cache" in s:
        return s["cache"][b, j]
    return s["pool"][s["page_table"].clamp(min=0)[b, j // PAGE], j % PAGE]


def plain_attend(s):
    case = s["case"]
    j, fine = positions(case, s["seq_lens"], case["hi"])
    rows = gather(s, j)
    rows = dequantise(rows, case["unit"]) if case["op"] == "packed" else rows.float()
    o, lse = attend(s["qt"].float(), rows, visible(case, s["seq_lens"], j, fine))
    return o.to(torch.bfloat16), lse


def plain_append(s):
    B, Q = s["case"]["B"], s["case"]["Q"]
    j = s["start"][:, None] + torch.arange(Q, device="cuda")
    page = torch.gather(s["page_table"], 1, (j // PAGE).long())
    packed = quantise(s["rows"].float(), s["case"]["unit"])
    s["pool"][page, j % PAGE] = packed
    s["seq_lens"].copy_(s["start"] + Q)
    return dequantise(s["pool"][page, j % PAGE], s["case"]["unit"]).to(torch.bfloat16), s["seq_lens"]


def free_pages(refs, n):
    """The n lowest free pages, in order."""
    return (refs == 0).nonzero().squeeze(1)[:n]


def plain_release(table, lens, refs):
    k = torch.arange(table.shape[1], device="cuda")
    go = (table >= 0) & (k[None] >= -(-lens.long() // PAGE)[:, None])
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -go.flatten().to(torch.int32))
    table.masked_fill_(go, -1)


def plain_fork(pool, table, lens, refs, parents, children):
    L = lens[parents.long()]
    rows = table[parents.long()]
    k = torch.arange(table.shape[1], device="cuda")
    full = k[None] < (L.long() // PAGE)[:, None]
    part = k[None] * PAGE < L.long()[:, None]
    part = part & ~full
    old = rows[part].long()
    new = free_pages(refs, old.numel())
    pool[new] = pool[old]
    shared = rows[full].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    refs[new] = 1
    rows = torch.where(full, rows, -1)
    rows[part] = new.to(torch.int32)
    table[children.long()] = rows
    lens[children.long()] = L


def plain_reserve(pool, table, lens, refs, Q):
    k = torch.arange(table.shape[1], device="cuda")
    need = (k[None] >= (lens.long() // PAGE)[:, None]) & (k[None] <= ((lens.long() + Q - 1) // PAGE)[:, None])
    copy = need & (table >= 0) & (refs[table.clamp(min=0).long()] > 1)
    take = (need & (table < 0)) | copy
    new = torch.full_like(table, -1)
    new[take] = free_pages(refs, int(take.sum())).to(torch.int32)
    old = table[copy].long()
    pool[new[copy].long()] = pool[old]
    refs.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    refs[new[take].long()] = 1
    table.copy_(torch.where(take, new, table))


def plain_compact(pool, table, refs):
    used = refs > 0
    n = used.sum()
    p = torch.arange(refs.numel(), device="cuda")
    src = (used & (p >= n)).nonzero().squeeze(1)
    dst = (~used & (p < n)).nonzero().squeeze(1)
    pool[dst] = pool[src]
    to = p.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    return n.to(torch.int32).view(1)


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "append":
        s["seq_lens"].copy_(s["start"])
    elif op in ("beam", "compact"):  # the step starts from the same bookkeeping every time
        s["page_table"].copy_(s["table0"])
        s["seq_lens"].copy_(s["lens0"])
        s["refs"].copy_(s["refs0"])
    if op == "beam":
        s["seq_lens"].index_fill_(0, s["children"].long(), 0)  # the sequences that end
    if not own:
        if op in ("window", "packed"):
            return plain_attend(s)
        if op == "append":
            return plain_append(s)
        pool, table, lens, refs = s["pool"], s["page_table"], s["seq_lens"], s["refs"]
        if op == "beam":
            plain_release(table, lens, refs)
            plain_fork(pool, table, lens, refs, s["parents"], s["children"])
            plain_reserve(pool, table, lens, refs, case["Q"])
            return table, lens, refs, pool
        return table, refs, plain_compact(pool, table, refs), pool
    import mla_absorbed_latent_mtp_b200 as m
    if op == "window" and not case["paged"]:
        return m.mla_attend_window_dense(s["qt"], s["cache"], case["window"], case["sinks"], s["seq_lens"],
                                         workspace=s["workspace"], status=s["status"])
    if op == "window":
        return m.mla_attend_window_paged(s["qt"], s["pool"], s["page_table"], s["seq_lens"], case["window"], case["sinks"],
                                         workspace=s["workspace"], status=s["status"])
    if op == "packed":
        return m.mla_attend_packed(s["qt"], s["pool"], s["page_table"], s["seq_lens"], unit=case["unit"], window=case["window"],
                                   sinks=case["sinks"], workspace=s["workspace"], status=s["status"])
    if op == "append":
        m.mla_cache_append_packed(s["pool"], s["page_table"], s["seq_lens"], s["rows"], unit=case["unit"], status=s["status"])
        rows = m.mla_cache_unpack(s["pool"], s["page_table"], s["start"], case["Q"], unit=case["unit"], status=s["status"])
        return rows, s["seq_lens"]
    pool, table, lens, refs = s["pool"], s["page_table"], s["seq_lens"], s["refs"]
    if op == "beam":
        m.mla_pages_release(table, lens, refs, status=s["status"])
        m.mla_pages_fork(pool, table, lens, refs, s["parents"], s["children"], workspace=s["workspace"], status=s["status"])
        m.mla_pages_reserve(pool, table, lens, refs, case["Q"], workspace=s["workspace"], status=s["status"])
        return table, lens, refs, pool
    return table, refs, m.mla_pages_compact(pool, table, refs, workspace=s["workspace"], status=s["status"]), pool


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, B = case["op"], case["B"]
    mean = (case["lo"] + case["hi"]) / 2
    if op in ("window", "packed"):
        Q = case["Q"]
        seen = read = mean
        if case["window"]:
            seen = min(mean, case["window"] + case["sinks"])
            read = min(mean, case["window"] + case["sinks"] + Q - 1)
        row = R * 2 if op == "window" else ROW_BYTES
        return dict(bytes=B * read * row + B * Q * H * (R * 4 + 4), flops=4.0 * B * Q * H * R * seen)
    if op == "append":
        rows = B * case["Q"]  # rows in, packed rows out; packed rows in, values out
        return dict(bytes=rows * (R * 2 + 2 * ROW_BYTES + R * 2), flops=0)
    page = PAGE * (ROW_BYTES if case["packed"] else R * 2)
    max_pages = -(-(case["hi"] + case.get("Q", 0)) // PAGE) + 1
    books = 4 * B * max_pages
    if op == "beam":
        return dict(bytes=2 * page * case["forks"] * 63 / 64 + 6 * books, flops=0)
    used = B * case["keep"] * (mean / PAGE + 0.5)
    moved = used * max(0.0, 1 - used / (B * max_pages))
    return dict(bytes=2 * page * moved + 4 * books, flops=0)


# ----------------------------------------------------------------------------- in 64 bits
def _exact_values(packed, unit):
    """Packed bytes -> float64 values, by the fields of the two formats."""
    low, high = packed[..., : R // 2].long() % 16, packed[..., : R // 2].long() // 16
    code = torch.stack([low, high], -1).flatten(-2)
    e, f = code % 8 // 2, code % 2
    mag = torch.where(e == 0, f * 0.5, (1 + f * 0.5) * torch.exp2((e - 1).double()))
    v = torch.where(code >= 8, -mag, mag).double()
    sc = packed[..., R // 2 :].long()
    e, f = sc % 128 // 8, sc % 8
    s = torch.where(e == 0, f * 2.0**-9, (1 + f / 8.0) * torch.exp2((e - 7).double())).double()
    return v * s.repeat_interleave(GROUP, -1) * unit


def _nearest_even(x, step):
    return torch.round(x / step) * step


def exact(case, seed):
    if case["op"] in ("beam", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        y = (s["rows"].double() / case["unit"]).unflatten(-1, (R // GROUP, GROUP))
        a = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
        exponent = torch.floor(torch.log2(a.clamp(min=2.0**-6)))
        scale = _nearest_even(a, torch.exp2(exponent - 3)).clamp(max=448.0)
        q = torch.where(scale > 0, y / scale.clamp(min=2.0**-9), 0.0).clamp(-6, 6)
        exponent = torch.floor(torch.log2(q.abs().clamp(min=1.0)))
        return (_nearest_even(q, torch.exp2(exponent - 1)) * scale).flatten(-2) * case["unit"], None
    B, Q = case["B"], case["Q"]
    o = torch.zeros(B, Q, H, R, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["seq_lens"].tolist()):
        for i in range(Q):
            t = L - Q + i
            j = torch.arange(t + 1, device="cuda")
            if case["window"]:
                j = j[(t - j < case["window"]) | (j < case["sinks"])]
            if j.numel() == 0:
                continue
            if "cache" in s:
                rows = s["cache"][b, j].double()
            else:
                rows = s["pool"][s["page_table"][b, j // PAGE].long(), j % PAGE]
                rows = _exact_values(rows, case["unit"]) if case["op"] == "packed" else rows.double()
            score = s["qt"][b, i].double() @ rows.T / 16
            lse[b, i] = torch.logsumexp(score, -1)
            o[b, i] = torch.exp(score - lse[b, i][:, None]) @ rows
    return o, lse
