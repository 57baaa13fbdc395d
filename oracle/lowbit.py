"""fp64 definitions of the low-bit operators (E4M3 activations and block-scaled
products, the 4-bit latent cache, attention over it), in numpy, written from
the formats themselves: values are picked from tables of every representable
number, so no rounding or conversion routine of a library takes part.
"""
from __future__ import annotations

import numpy as np
import torch

LATENT, ROPE, GROUP, BLOCK = 512, 64, 16, 128
ROW_BYTES = 416
SCALE = 192.0 ** -0.5


def _e4m3_table() -> np.ndarray:
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[b] = np.nan if (b & 0x7F) == 0x7F else (-v if b & 0x80 else v)
    return t


E4M3 = _e4m3_table()
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
_E4M3_POS = E4M3[:127]  # 0 .. 448, ascending; the index is the code


def _nearest(mag: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the value of `grid` (ascending, index = code) nearest to each magnitude; ties to the even code;
    magnitudes past the end take the last."""
    hi = np.clip(np.searchsorted(grid, mag), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = mag - grid[lo], grid[hi] - mag
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up | (mag >= grid[hi]), hi, lo)


def to_f64(x: torch.Tensor) -> np.ndarray:
    return x.detach().cpu().to(torch.float64).numpy()


def quantize_fp8(x: np.ndarray):
    """x [rows, cols] -> (code bytes, scales) of sga_quantize_fp8."""
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), dtype=np.uint8)
    scale = np.ones((rows, kb))
    largest = float(torch.finfo(torch.bfloat16).max)
    for j in range(kb):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        mag = np.minimum(np.where(np.isnan(part), 0.0, np.abs(part)), largest)
        for r in range(rows):
            top = mag[r].max()
            if top == 0:
                continue
            e = -126
            while top > 448.0 * 2.0 ** e:
                e += 1
            scale[r, j] = 2.0 ** e
        mag = np.minimum(np.abs(part) / scale[:, j:j + 1], 448.0)
        code = _nearest(np.where(np.isnan(mag), 0.0, mag), _E4M3_POS) + 128 * np.signbit(part)
        codes[:, j * BLOCK:(j + 1) * BLOCK] = np.where(np.isnan(part), 0x7F, code)
    return codes, scale


def block_scaled(codes: np.ndarray, scale: np.ndarray, rows_per_scale: int) -> np.ndarray:
    """The values of E4M3 code bytes [r, k] with scale [ceil(r / rows_per_scale), ceil(k / 128)]."""
    r, k = codes.shape
    s = np.repeat(np.repeat(scale, rows_per_scale, 0)[:r], BLOCK, 1)[:, :k]
    return E4M3[codes] * s


def kv4_pack(rows: np.ndarray):
    """rows [n, 576] -> (codes [n, 512] 0..15, scale bytes [n, 32], rope [n, 64])."""
    n = rows.shape[0]
    lat = rows[:, :LATENT].reshape(n, LATENT // GROUP, GROUP)
    nan = np.isnan(lat).any(-1)
    mag = np.abs(np.where(np.isnan(lat), 0.0, lat))
    scale = _nearest(mag.max(-1) / 6.0, _E4M3_POS)
    s = E4M3[scale][..., None]
    q = np.divide(mag, s, out=np.zeros_like(mag), where=s > 0)
    code = _nearest(q, E2M1) + 8 * np.signbit(lat)
    code[nan] = 0
    scale = np.where(nan, 0x7F, scale)
    return code.reshape(n, LATENT).astype(np.uint8), scale.astype(np.uint8), rows[:, LATENT:]


def kv4_values(packed: np.ndarray) -> np.ndarray:
    """Cache bytes [..., 416] -> values [..., 576]."""
    byte = packed[..., :LATENT // 2]
    code = np.stack([byte & 15, byte >> 4], -1).reshape(*packed.shape[:-1], LATENT)
    scale = np.repeat(E4M3[packed[..., 256:288]], GROUP, -1)
    lat = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7] * scale
    half = packed[..., 288:416].reshape(*packed.shape[:-1], ROPE, 2).astype(np.uint32)
    rope = ((half[..., 0] | (half[..., 1] << 8)) << 16).view(np.float32).astype(np.float64)
    return np.concatenate([lat, rope], -1)


def attend_kv4(q: np.ndarray, packed: np.ndarray, idx: np.ndarray, gate):
    """q [B,T,64,576], packed [B,L,416], idx [B,T,K], gate [B,T,64] or None ->
    (out [B,T,64,512], and what bounds its error: the same sum with |values|, the largest sum |q||k| * scale of a
    head, and the sum of the selected rows' |values|)."""
    B, T = q.shape[:2]
    out = np.zeros((B, T, q.shape[2], LATENT))
    spread = np.zeros_like(out)
    total = np.zeros_like(out)
    zabs = np.zeros((B, T, q.shape[2], 1))
    for b in range(B):
        for t in range(T):
            sel = idx[b, t][idx[b, t] >= 0]
            if not len(sel):
                continue
            rows = kv4_values(packed[b, sel])
            z = q[b, t] @ rows.T * SCALE
            zabs[b, t, :, 0] = (np.abs(q[b, t]) @ np.abs(rows.T)).max(-1) * SCALE
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            g = 1.0 if gate is None else (1 / (1 + np.exp(-gate[b, t])))[:, None]
            out[b, t] = p @ rows[:, :LATENT] * g
            spread[b, t] = p @ np.abs(rows[:, :LATENT]) * g
            total[b, t] = np.abs(rows[:, :LATENT]).sum(0)
    return out, spread, zabs, total


# ----------------------------------------------------------------------------- one layer in few bits
def _quantised(x: np.ndarray) -> np.ndarray:
    """The values that quantize_fp8 keeps of x [..., k]."""
    flat = x.reshape(-1, x.shape[-1])
    codes, scale = quantize_fp8(flat)
    return block_scaled(codes, scale, 1).reshape(x.shape)


def layer_forward(h, q_pos, packed, k_idx_cache, wts: dict, k: int = 2048, n_threads: int = 0, idx=None) -> dict:
    """The layer of sga_layer_forward_fp8kv4 in fp64, every activation between two contractions rounded to bf16.

    packed [B,L,416] bytes and k_idx_cache [B,L,128] are updated copies in the result; wts as layer_forward_fp8kv4
    takes them.  The attention is over `idx` [B,T,k], or over all positions 0..q_pos (at most k); what the indexer scores
    with (q_idx, w and the keys) is in the result."""
    from . import layer

    def weights(name):
        return block_scaled(wts[name].view(torch.uint8).cpu().numpy(), to_f64(wts[name + "_scale"]), 128)

    rb = layer.round_bf16
    w_hq, w_cq, w_o = weights("w_hq"), weights("w_cq"), weights("w_o")
    R = w_cq.shape[1]
    rp = -(-R // BLOCK) * BLOCK
    H, pos = _quantised(to_f64(h)), q_pos.cpu().numpy().astype(np.int64)
    B, T = pos.shape
    g1 = H @ w_hq.T
    c_q = rb(g1[..., :R])
    kv_row = np.concatenate([rb(g1[..., rp:rp + LATENT]),
                             rb(layer.rope(rb(g1[..., rp + LATENT:rp + LATENT + ROPE]), pos))], -1)
    k_row = rb(g1[..., rp + 640:rp + 768])
    g2 = _quantised(c_q) @ w_cq.T
    heads = g2[..., :12288].reshape(B, T, 64, 192)
    q_rope = rb(layer.rope(rb(heads[..., 128:]), pos[..., None]))
    q = np.concatenate([rb(np.einsum("bthd,hdj->bthj", rb(heads[..., :128]), to_f64(wts["w_uk"]))), q_rope], -1)
    gate = rb(g2[..., 12288:12352])
    packed, k_idx = packed.cpu().numpy().copy(), to_f64(k_idx_cache).copy()
    code, scale, rope_v = kv4_pack(kv_row.reshape(B * T, -1))
    bits = layer.bf16_bits(rope_v).view(np.uint8).reshape(B * T, 128)
    rows = np.concatenate([code[:, 0::2] | (code[:, 1::2] << 4), scale, bits], 1).reshape(B, T, ROW_BYTES)
    dense = np.full((B, T, k), -1, dtype=np.int32)
    for b in range(B):
        for t in range(T):
            packed[b, pos[b, t]], k_idx[b, pos[b, t]] = rows[b, t], k_row[b, t]
            if idx is None:
                dense[b, t, :pos[b, t] + 1] = np.arange(pos[b, t] + 1)
    idx = dense if idx is None else idx
    out = rb(attend_kv4(q, packed, idx, gate)[0])
    o = rb(np.einsum("bthj,hij->bthi", out, to_f64(wts["w_uv"]))).reshape(B, T, -1)
    return {"idx": idx, "packed": packed, "k_idx": k_idx, "y": _quantised(o) @ w_o.T,
            "q_idx": rb(g2[..., 12416:]).reshape(B, T, 64, 128), "w": rb(g1[..., rp + 768:])}
