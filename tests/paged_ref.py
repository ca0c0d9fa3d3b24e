"""The paged cache operators in 64 bits on the CPU, from their definitions, and the pools the
tests run them on."""
import math

import torch

NEG = -math.inf


def make_pool(lens, page_size, Hkv, D, dtype, seed=0, spare=3, layout="page_head_row", poison=True, width=None):
    """A pool whose sequences' pages are scattered, with NaN wherever no sequence has a
    position: behind each end, and in the pages that nobody holds.  Returns (k, v, table) on
    the CPU; table entries behind a sequence's last page are out of the pool on purpose."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page_size) for n in lens]
    n_pages = sum(pages) + spare
    k = torch.randn(n_pages, Hkv, page_size, D, generator=g).to(dtype)
    v = torch.randn(n_pages, Hkv, page_size, D, generator=g).to(dtype)
    perm = torch.randperm(n_pages, generator=g)
    width = max(1, max(pages)) if width is None else width
    table = torch.full((len(lens), width), 10 ** 9, dtype=torch.int32)
    held = torch.zeros(n_pages, page_size, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = perm[at:at + pages[b]].to(torch.int32)
        for j in range(pages[b]):
            held[perm[at + j], :min(page_size, n - j * page_size)] = True
        at += pages[b]
    if poison:
        hole = ~held[:, None, :, None].expand_as(k)
        k[hole] = math.nan
        v[hole] = math.nan
    order = {"page_head_row": (0, 1, 2, 3), "page_row_head": (0, 2, 1, 3), "head_page_row": (1, 0, 2, 3)}[layout]
    back = [order.index(i) for i in range(4)]
    k, v = (t.permute(order).contiguous().permute(back) for t in (k, v))
    return k, v, table


def to_gpu(t):
    """The tensor on the GPU with the same strides (a permuted view stays one)."""
    order = sorted(range(t.dim()), key=lambda i: -t.stride(i))
    return t.permute(order).contiguous().cuda().permute([order.index(i) for i in range(t.dim())])


def positions(n, page_size, n_meta=0, window=0, pages=None):
    """Visible positions of a sequence of n, ascending (list order for a page list)."""
    if pages is not None:
        total = -(-n // page_size)
        pages = [j for j in pages[:total] if 0 <= j < total]
        return [p for j in pages for p in range(j * page_size, min(n, (j + 1) * page_size))]
    return [p for p in range(n) if window == 0 or p < n_meta or p >= n - window]


def attention(k, v, table, lens, q, scale, n_meta=0, window=0, page_idx=None):
    """(out, lse, size): size[b, h] bounds sum_d |q_d k_d| * scale over the visible keys."""
    B, Hq, D = q.shape
    Hkv, ps = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), NEG, dtype=torch.float64)
    size = torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        for g in range(Hkv):
            pos = positions(lens[b], ps, n_meta, window, None if page_idx is None else page_idx[b, g].tolist())
            if not pos:
                continue
            pos = torch.tensor(pos)
            page = table[b].long()[pos // ps]
            kk, vv = k[page, g, pos % ps].double(), v[page, g, pos % ps].double()
            h = slice(g * G, (g + 1) * G)
            x = q[b, h].double() @ kk.T * scale
            lse[b, h] = torch.logsumexp(x, -1)
            out[b, h] = torch.exp(x - lse[b, h, None]) @ vv
            size[b, h] = (q[b, h].double().abs() @ kk.abs().T).amax(-1) * abs(scale)
    return out, lse, size


def rotate(x, pos, base):
    """Half-split rotation of x [T, heads, D] by pos * base^(-2j/D)."""
    x = x.double()
    if base == 0:
        return x
    h = x.shape[-1] // 2
    ang = torch.tensor(pos, dtype=torch.float64)[:, None] * torch.tensor(
        [base ** (-j / h) for j in range(h)], dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def scores(k_lo, k_hi, pages, q):
    """Page scores [Hkv, n] of one sequence: per head the maximum over the box, summed."""
    Hkv, D = k_lo.shape[1:]
    qg = q.double().view(Hkv, -1, 1, D)
    lo, hi = (t[pages.long()].double().transpose(0, 1)[:, None] for t in (k_lo, k_hi))
    return torch.maximum(qg * lo, qg * hi).sum(-1).sum(1)


def select(score, n_first, n_last, top):
    """Ascending page numbers of one (sequence, head), -1 behind the last."""
    n = len(score)
    forced = {j for j in range(n) if j < n_first or j >= n - n_last}
    rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-score[j], j))
    pick = range(n) if n <= top else sorted(list(forced) + rest[:top - len(forced)])
    return list(pick) + [-1] * (top - len(pick))
