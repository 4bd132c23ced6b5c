"""The rotary frequencies in 80 decimal digits, as turns per position in fixed point. Test infrastructure only."""
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, localcontext

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turns(bits=64, base=10000.0, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """The 32 integers nearest to 2^bits f_i / (2 pi)."""
    out = []
    with localcontext() as ctx:
        ctx.prec = 80
        base, factor, ln = Decimal(base), Decimal(factor), Decimal(base).ln()
        for i in range(32):
            f = (-ln * i / 32).exp()
            share = Decimal(1)
            if original_len:
                pair_of = lambda n: 32 * (original_len / (Decimal(n) * 2 * PI)).ln() / ln  # noqa: E731
                clamp = lambda v: min(max(v, Decimal(0)), Decimal(63))  # noqa: E731
                low = clamp(pair_of(beta_fast).to_integral_value(ROUND_FLOOR))
                high = clamp(pair_of(beta_slow).to_integral_value(ROUND_CEILING))
                high = high if high > low else low + Decimal("0.001")
                share = min(max((i - low) / (high - low), Decimal(0)), Decimal(1))
            f = f * (1 - share) + f / factor * share
            out.append(int((f / (2 * PI) * 2 ** bits).to_integral_value()))
    return out


def angles(pos, **kw):
    """Angles in radians (floats in [0, 2 pi)) of integer positions, reduced exactly: [positions][32]."""
    t = turns(160, **kw)
    return [[float(Decimal((int(p) * v) % (1 << 160)) / (1 << 160)) * float(2 * PI) for v in t] for p in pos]
