"""Plain references of 4-bit pages on the CPU: codes and scales by search over all their values, the layout of a page,
and problems of attention over them. Written from the definitions in include/mkv.h; no code of the library is used."""
import numpy as np
import torch

import geometric_kv_cache_gb300 as mkv
import paged_util as pu
from test_gpu_paged_attention import Problem

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda"

# every value of the two types, by code
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def nearest(x, values):
    """Codes of the values nearest to x >= 0 (fp32, taken exactly), ties to the even code, saturated."""
    x = np.minimum(x.astype(np.float64), values[-1])
    hi = np.searchsorted(values, x).clip(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - x, x - values[lo]  # exact: neighbours of few bits
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)


def encode(x, scale):
    """x fp32 [..., d] (finite) as codes uint8 [..., d / 2] and scales uint8 [..., d / 16]."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, 16)
    inv, inv6 = np.float32(1.0 / float(np.float32(scale))), np.float32(1.0 / (6.0 * float(np.float32(scale))))
    with np.errstate(all="ignore"):
        s = nearest(np.abs(g).max(-1) * inv6, E4M3)
        v = E4M3[s].astype(np.float32)
        r = np.where(s == 0, np.float32(0), inv / v).astype(np.float32)
        t = g * r[..., None]
    c = nearest(np.abs(t), E2M1)
    c = c | ((t < 0) & (c > 0)).astype(np.uint8) << 3
    c = c.reshape(*x.shape)
    return torch.from_numpy(c[..., 0::2] | c[..., 1::2] << 4), torch.from_numpy(s)


def decode(codes, scales):
    """fp64 [..., d]; a scale of NaN gives NaN."""
    c = np.stack([codes.numpy() & 15, codes.numpy() >> 4], -1).reshape(*codes.shape[:-1], -1)
    x = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.append(E4M3, np.nan)[scales.numpy() & 127]
    return torch.from_numpy((x.reshape(*s.shape, 16) * s[..., None]).reshape(x.shape))


def to_pages(codes, scales):
    """uint8 [n_pages, page, d * 9 / 16] of codes [n_pages, page, d / 2] and scales [n_pages, page, d / 16]."""
    n, page = codes.shape[:2]
    return torch.cat([codes.flatten(1), scales.flatten(1)], 1).view(n, page, -1).contiguous()


def from_pages(pages):
    n, page, b = pages.shape
    flat = pages.flatten(1)
    return flat[:, :page * b * 8 // 9].view(n, page, -1), flat[:, page * b * 8 // 9:].view(n, page, -1)


def rows_of(pages):
    """Token rows of codes and scales together [n_pages, page, d * 9 / 16], in a type that paged_util takes for bytes."""
    return torch.cat(from_pages(pages), -1).view(F8)


def rows_to_pages(rows):
    b = rows.shape[-1]
    return to_pages(rows.view(torch.uint8)[..., :b * 8 // 9].contiguous(), rows.view(torch.uint8)[..., b * 8 // 9:].contiguous())


def random_pages(seed, n_pages, page, d):
    k, v = pu.random_pool(seed, n_pages, page, d, BF)
    return to_pages(*encode(k.float(), 1.0)), to_pages(*encode(v.float(), 1.0))


class Four(Problem):
    """Problem over 4-bit pages: k and v hold their values as bf16 (exact), kp and vp the pages. Rows that no list
    reaches have NaN scales. `dtype` is E4M3's for the bounds: weights are fp16 next to both."""

    def __init__(self, *args, **kw):
        super().__init__(*args[:6], BF, *args[6:], **kw)
        self.dtype, self.scales = F8, (0.75, 1.25)
        both = []
        for x in (self.k, self.v):
            unused = x.isnan().any(-1)
            codes, scales = encode(x.float().nan_to_num(0.0), 1.0)
            codes[unused], scales[unused] = 0xFF, 0x7F
            both.append((to_pages(codes, scales), decode(codes, scales).to(BF)))
        (self.kp, self.k), (self.vp, self.v) = both

    def on_device(self, strided=False):
        Q = self.Q.to(DEV)
        O = torch.full_like(Q, 7.0)
        if strided:  # slices of wider rows
            wide = torch.full((self.n, Q.shape[1] + 3, self.d), 3.0, dtype=BF, device=DEV)
            wide[:, 1:-2] = Q
            Q, O = wide[:, 1:-2], torch.full_like(wide, 7.0)[:, 2:-1]
        lse = torch.full(Q.shape[:2], 7.0, device=DEV)
        return (Q, *(x.to(DEV) for x in (self.kp, self.vp, self.table, self.lens, self.start)), O, lse)

    def run(self, window=0, sinks=0, scale=None, max_q=None, strided=False):
        Q, k, v, table, lens, start, O, lse = self.on_device(strided)
        max_q = self.max_q if max_q is None else max_q
        ws = mkv.attention_workspace_for(Q, k, table, max_q, self.max_len)
        ws[256:] = 255  # (what a call leaves in the workspace is NaN to the next)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start, max_q, self.max_len, O, ws, scale=scale,
                                k_scale=self.scales[0], v_scale=self.scales[1], window=window, sinks=sinks, lse=lse)
        self.status = mkv.mkv_device_status(ws)
        assert int(ws[:256].sum()) == 0
        return O.cpu(), lse.cpu()


    def check(self, O, lse, window=0, sinks=0, scale=None, rows=None):
        """Problem.check, its reference list by list in matrices."""
        n, hq, d = self.Q.shape
        scale = d ** -0.5 if scale is None else scale
        ref, A, W = (torch.zeros((n, hq, d), dtype=torch.float64) for _ in range(3))
        ref_lse, E = torch.full((n, hq), -np.inf, dtype=torch.float64), torch.zeros((n, hq), dtype=torch.float64)
        for b in range(self.lens.shape[0]):
            t0, t1 = int(self.start[b]), int(self.start[b + 1])
            for j in range(self.lens.shape[1]):
                L, h = int(self.lens[b, j]), slice(j * self.G, (j + 1) * self.G)
                K, V = (pu.rows_of(x, self.table[b, j], L, self.page) * s for x, s in zip((self.k, self.v), self.scales))
                own, key = L - (t1 - t0) + torch.arange(t1 - t0)[:, None], torch.arange(L)[None]
                hidden = key > own
                if window:
                    hidden |= (key <= own - window) & (key >= sinks)
                some = ~hidden.all(1)
                if not some.any():
                    continue
                hidden, q = hidden[some][:, None], self.Q[t0:t1, h].double()[some]
                x = (q @ K.T * scale).masked_fill(hidden, -np.inf)
                w = torch.exp(x - x.amax(-1, keepdim=True))
                l = w.sum(-1, keepdim=True)
                at = torch.arange(t0, t1)[some]
                ref[at, h], A[at, h], W[at, h] = w @ V / l, w @ V.abs() / l, (~hidden).double() @ V.abs() / l
                ref_lse[at, h] = x.amax(-1) + torch.log(l[..., 0])
                E[at, h] = (q.abs() @ K.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(-1)
        tol, tol_lse = pu.attention_bounds(ref, ref_lse, A, W, E, d, self.dtype)
        end = int(self.start[-1])
        rows = slice(0, end) if rows is None else rows
        err = (O.double() - ref).abs()
        bad = ~(err <= tol)
        assert not bad[rows].any(), (int(bad[rows].sum()), float((err / tol)[rows].max()))
        assert torch.equal(torch.isinf(lse)[rows], torch.isinf(ref_lse)[rows])
        off = (lse.double() - ref_lse).abs()
        assert not (off > tol_lse)[rows][torch.isfinite(ref_lse[rows])].any(), float(off[rows].nan_to_num(0).max())
        assert torch.equal(O[end:], torch.full_like(O[end:], 7.0)) and torch.equal(lse[end:], torch.full_like(lse[end:], 7.0))


def wide(seed, counts, extra, G, d, page, heads=16, **kw):
    """A problem of enough query rows for the form for chunks: its parts in the workspace are 128 or 256 rows."""
    p = Four(seed, counts, [[max(0, c + extra[(b + j) % len(extra)]) for j in range(heads)] for b, c in enumerate(counts)],
             G, d, page, **kw)
    ws = mkv.attention_workspace_for(torch.empty((p.n, heads * G, d), dtype=BF, device=DEV), p.kp.to(DEV),
                                     torch.empty(p.table.shape, dtype=torch.int32, device=DEV), p.max_q, p.max_len)
    assert ws.numel() > 152 * 2 * 100 * (4 * d + 8)
    return p
