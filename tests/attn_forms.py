"""Shapes that reach every form of the attention's kernels: many short items for
workgroups that own 128 frames, fewer for 64, a few for 32, and few queries of
heads that share their keys; every padded head width, filled and not, with whole
groups of 8 elements and without; lengths, windows, positions, biases and shared
key heads in turn."""

# (owned frames in units of 32, B, H, Hkv, frames)
SIZES = [(4, 50, 16, 8, 140), (2, 23, 4, 2, 140), (1, 3, 4, 2, 140)]
HEADS = [32, 24, 20, 64, 40, 50, 96, 72, 90, 128, 104, 127]


def _options(n, B, T):
    ragged = [max(1, T - (5 * b) % (T - 9)) for b in range(B)]
    return [dict(q_len=ragged, k_len=ragged),
            dict(q_len=ragged, k_len=ragged, left=30, right=11),
            dict(left=60, right=0),
            dict(q_len=ragged, k_len=ragged, bias=False),
            dict(k_len=ragged, reach=20, special=True),
            dict(more_keys=21, pos=[b % 22 for b in range(B)], reach=128)][n % 6]


def self_attention():
    """For both directions."""
    cases, n = [], 0
    for own, B, H, Hkv, T in SIZES:
        for D in HEADS:
            for elem in (2, 4):
                o = _options(n, B, T)
                if elem == 4 and D > 64 and own == 1 and o.get("reach", 40) > 40:
                    o["reach"] = 40  # LDS holds no more beside the widest tiles
                cases.append(dict(B=B, Tq=T, Tk=T + o.pop("more_keys", 0), H=H, Hkv=Hkv, D=D, elem=elem, own=own, **o))
                n += 1
            n += 1
    # frames that do not lie next to each other, on 16-byte chunks and off them; the largest reach at the widest heads
    for elem in (2, 4):
        for own, B, H, Hkv, T in SIZES:
            cases.append(dict(B=B, Tq=T, Tk=T, H=H, Hkv=Hkv, D=64, elem=elem, own=own, pad=3))
            cases.append(dict(B=B, Tq=T, Tk=T, H=H, Hkv=Hkv, D=96, elem=elem, own=own, pad=8))
            cases.append(dict(B=B, Tq=T, Tk=T, H=H, Hkv=Hkv, D=128, elem=elem, own=own, reach=1024))
    return cases


def few_queries():
    """For the forward: the heads of a group side by side, and not."""
    return [dict(B=3, Tq=3, Tk=300, H=8, Hkv=Hkv, D=D, elem=elem, own=1, k_len=[300, 5, 131], pos=[297, 0, 100])
            for D in HEADS for elem in (2, 4) for Hkv in (2, 8)]


def line(c):
    """The case as the plan's program reads it."""
    reach = c.get("reach", 40) if c.get("bias", True) else 0
    return " ".join(str(v) for v in (c["elem"], c["B"], c["Tq"], c["Tk"], c["H"], c["Hkv"], c["D"], reach, c.get("left", -1),
                                     c.get("right", -1), c.get("pad", 0)))


def name(c):
    return "-".join(str(c[n]) for n in ("own", "D", "elem")) + "".join(
        f"-{k}" for k in ("left", "pos", "special", "pad", "reach") if k in c) + ("" if c.get("bias", True) else "-flat") + (
        f"-{c['Hkv']}" if c["Tq"] < 32 else "")
