"""The error of attention by its norm.

Over a long context the outputs shrink like one over the root of its length, while a bound from the sum of
p |v| does not, so that a lost part of the context stays below it.  The norm of the error tells."""
import math


def norm_error(got, want):
    return float((got - want).norm() / want.norm())


def norm_limit(elements):
    """For `elements` outputs over contexts of some thousand positions and values around zero.

    A rounding to BF16 is off by a uniform share of at most 2^-8 of the value, 2^-8 / sqrt 3 in the mean square.
    Two of them count: the output's own, and those of the p: the errors d_j p_j v_j add up like the p_j v_j do,
    both around zero, so their norms are as d_j to one.  The quotient of two norms of that many terms strays by
    1 / sqrt(elements); five times that is allowed."""
    return 2.0 ** -8 * math.sqrt(2 / 3) * (1 + 5 / math.sqrt(elements))
