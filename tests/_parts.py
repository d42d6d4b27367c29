"""How far fp32 products of three bf16 parts may be off, as a root mean square
relative to the result's.

A factor is a1 + a2 + a3, each part the nearest bf16 number to what is left (rms
of a2 1.6e-3 of a, of a3 2^-8 of that).  Six of the nine products of parts are
summed, 128 of K at a time in the tensor core, the five small ones first: only
the last 8 additions of 16 products each (a1 b1; for `pairs` products in one sum
8 times as many) are of the sum's own size.  An addition there drops less than
2^-23 of the running sum, which grows like the root of its length: over n of them
sum sqrt(j / n) = 2 n / 3 + 1/2.  All drops go towards zero, so they add up.  The
sums of 128 are added in fp32, each addition off by 2^-24 at most of a sum that
grows in the same way.  The three products left out come to 2e-8.

A product of parts that is lost costs 2.8e-6 (a2 b2), 2.4e-6 (a1 b3, a3 b1) or
1.7e-3 (a1 b2, a2 b1).
"""
LEFT_OUT = 2e-8
TERMS = ((1, 1), (0, 2), (2, 0), (0, 1), (1, 0), (0, 0))


def rms(t):
    return t.double().square().mean().sqrt().item()


def tolerance(K, pairs=1):
    n = pairs * min(8, -(-K // 16))
    sums = -(-K // 128)
    return 2.0 ** -23 * (2 * n / 3 + 0.5) + 2.0 ** -24 * (2 * sums / 3 + 0.5) + LEFT_OUT


def parts(t):
    """Three bf16 numbers of each fp32 one, in 64 bits."""
    out, rest = [], t.double()
    for _ in range(3):
        out.append(rest.float().bfloat16().double())
        rest = rest - out[-1]
    assert not rest.any()
    return out


def product(a, b, terms=TERMS):
    """a @ b from the given products of parts, exact otherwise."""
    a, b = parts(a), parts(b)
    return sum(a[i] @ b[j] for i, j in terms)
