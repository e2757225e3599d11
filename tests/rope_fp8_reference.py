"""Plain float64 versions of the rotary append and of attention over the 8-bit
cache, on the CPU, token by token and tile by tile as the definitions say, and
the tolerances that the kernels' roundings allow.

Roundings (half a step: bf16 2^-8, f16 2^-11, fp32 2^-24, E4M3 2^-4 relative):
  * the rotation is one fp32 evaluation of x cos a - y sin a from an angle
    within 2^-24 of a turn (4e-7 rad), with cos and sin within 2 ulp: together
    below 2^-19 (|x| + |y|); then one rounding to bf16 or to an E4M3 code;
  * a logit is a dot product of 128 exact products summed in fp32 (in any
    order: at most 128 * 2^-24 of the sum of their magnitudes) with a few fp32
    factors, 140 * 2^-24 in all; 2^x is within 2^-22;
  * over the 8-bit cache a query entry is taken in f16, scaled by the power of
    two that brings the row's largest entry to [2^14, 2^15): bf16's 8 bits fit,
    and where f16 is subnormal it is off by at most 2^-25, 2^-39 of the largest;
  * a softmax weight rounds to f16 (2^-11 relative; 2^-25 of the largest weight
    below the type's normal range) over the 8-bit cache, to bf16 (2^-8) over
    the bf16 one; the weighted sum accumulates in fp32 over n tokens, and the
    output rounds to bf16.
"""
import math

import torch

TILE = 64
E4M3_MAX = 448.0


def rotate(x, pos, inv_freq, interleaved=False, pair_axis=None, scale=1.0):
    """x [tokens][heads][128] float64, pos int [axes][tokens] -> (rotated, slack of the fp32 evaluation)."""
    half = inv_freq.numel()
    axis = torch.zeros(half, dtype=torch.long) if pair_axis is None else pair_axis.long()
    ang = pos.double()[axis].t() * inv_freq.double()                    # [tokens][pairs]
    out, slack = x.clone(), torch.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = ang[:, i].cos()[:, None], ang[:, i].sin()[:, None]
        u, v = x[:, :, a], x[:, :, b]
        out[:, :, a] = (u * c - v * s) * scale
        out[:, :, b] = (v * c + u * s) * scale
        slack[:, :, a] = slack[:, :, b] = (u.abs() + v.abs()) * abs(scale) * 2.0 ** -19
    return out, slack


def places(table, lens, cu, block):
    """(sequence, position, page, slot) of every new token."""
    got = []
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            p = lens[s] - n + i
            got.append((s, p, int(table[s][p // block]), p % block))
    return got


def decode_e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def encode_e4m3(x):
    """float64 -> codes by torch's conversion (nearest even), saturated."""
    return x.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn).view(torch.uint8)


def need_of(top):
    e = -100
    while top > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_tiles(pool, scale, x, spots, cu):
    """The E4M3 append of float64 rows x [tokens][heads][128]: returns, per touched (page,
    tile): (first new slot, token ids, held scales, new scales [heads])."""
    tiles = {}
    for i, (s, p, pg, slot) in enumerate(spots):
        tiles.setdefault((pg, slot // TILE), []).append(i)
    done = {}
    for (pg, sub), ids in tiles.items():
        first = spots[ids[0]][3] - sub * TILE
        was = scale[pg, sub].double()
        need = torch.tensor([need_of(float(x[ids, h].abs().max())) for h in range(x.shape[1])], dtype=torch.float64)
        done[(pg, sub)] = (first, ids, was, need if first == 0 else torch.maximum(was, need))
    return done


def stored(codes, scale):
    """The values an 8-bit pool stands for, float64 [pages][block][heads][128]."""
    return decode_e4m3(codes) * scale.double().repeat_interleave(TILE, dim=1)[..., None]


def attention(q, k_pool, v_pool, table, block, q_seq, q_pos, sel, cnt, sm_scale, p_half=2.0 ** -11):
    """(out, lse, out tolerance, lse tolerance) in float64, query by query; q [T][Hq][128] and
    the pools' values float64; p_half: half a step of the softmax weights' type."""
    T, hq, _ = q.shape
    hkv = k_pool.shape[2]
    group = hq // hkv
    out, lse = torch.zeros_like(q), torch.full((T, hq), -math.inf, dtype=torch.float64)
    otol, ltol = torch.full_like(q, 1e-12), torch.full((T, hq), 1e-12, dtype=torch.float64)
    for t in range(T):
        toks = []
        for j in range(int(cnt[t])):
            b = int(sel[t][j])
            pg = int(table[q_seq[t]][b])
            for o in range(block):
                if b * block + o <= q_pos[t]:
                    toks.append((pg, o))
        if not toks:
            continue
        pg = torch.tensor([a for a, _ in toks])
        of = torch.tensor([b for _, b in toks])
        k, v, n = k_pool[pg, of], v_pool[pg, of], len(toks)              # [n][hkv][128]
        for h in range(hq):
            kh, vh, qh = k[:, h // group], v[:, h // group], q[t, h]
            s = kh @ qh * sm_scale
            top = s.max()
            w = (s - top).exp()
            norm = w.sum()
            out[t, h] = (w / norm) @ vh
            lse[t, h] = top + norm.log()
            delta = float((kh.abs() @ qh.abs()).max()) * sm_scale * 140 * 2.0 ** -24 + 2.0 ** -21
            delta += float(kh.abs().sum(1).max() * qh.abs().max()) * sm_scale * 2.0 ** -39
            mass = (w / norm) @ vh.abs()
            tiny = 2.0 ** -25 / norm * vh.abs().sum(0)
            otol[t, h] = out[t, h].abs() * 2.0 ** -8 + mass * (2 * delta + p_half + n * 2.0 ** -24) + tiny + 1e-30
            ltol[t, h] = delta + (n + 8) * 2.0 ** -24 + abs(float(lse[t, h])) * 2.0 ** -22
    return out, lse, otol, ltol
