"""The error that a product with integer 4-bit weights may have, from its definition: sums in fp32 of products that are
exact in fp32, times the group's scale in fp32, and the result rounded once to bf16.

A sum of k values in fp32, whatever the order of its additions and the instructions that make them, has an error of at
most (k - 1) u sum |x w| (first order), u = 2^-23 where a matrix instruction truncates.  A group's scale is one more
rounding; a kernel that keeps its sums in units of the scale's mantissa rounds a quotient and a product a group and one
at the end.  All together at most (k + 2 k / group + 4) u B, B = sum |x w|.

The kernels for few tokens sum x (c + q - z) over a group, c at most 192, and take the sum of c x off: at most group u
sum |x| (2 c + |q - z|) |s| over the groups, but nothing for a group with q = z everywhere, whose two sums are equal.

On top half a bf16 step of the result, 2^-20 of it all for the second order, and 2^-133 for bf16's own underflow."""
import numpy as np


def bound(ref, magnitude, k, group, offset=None):
    """Of |y - ref|; magnitude: sum |x w|; offset, for the kernels that have it: sum |x| (2 c + |q - z|) |s| over the groups
    that are not q = z everywhere."""
    e = (k + 2 * k / group + 4) * 2.0 ** -23 * magnitude
    if offset is not None:
        e = e + group * 2.0 ** -23 * offset
    return (2.0 ** -8 * (np.abs(ref) + e) + e) * (1 + 2.0 ** -20) + 2.0 ** -133
