"""Roundings that the layer operators' fp32 computations make, counted along their sums and recurrences
instead of by their lengths, for the tests that hold them close: an error of one part in a few thousand
(a value rounded to bf16 on the way) lies outside."""


def norm_depth(dim):
    """Additions on the longest path of a row's sum: a lane adds pieces of 8 values (two at least where a
    wave has a row, one for every 2048 values of a long row), then 6 levels over the wave, then up to 16
    waves one by one."""
    return 8 * max(2, -(-dim // 2048)) + 6 + 16


def rms_count(dim):
    """Roundings of 1 / sqrt(mean s^2 + eps): s itself and its square (3), the sum, the division and eps (2),
    halved by the root; the root's own unit in the last place (2) and a power of two."""
    return (norm_depth(dim) + 5) // 2 + 3


def norm_count(dim):
    """Of v = s r w, s rounded once, relative to v."""
    return rms_count(dim) + 3


def norm_bwd_count(dim):
    """Of dres + r (w dy - sh mean(w dy sh)), relative to the terms' magnitudes: sh has r's and one more; the
    mean has two products a value, the sum, r and two more; then three products and two sums."""
    return (rms_count(dim) + 1) + (2 + norm_depth(dim) + rms_count(dim) + 2) + rms_count(dim) + 5


def dweight_count(rows, dim):
    """Of the sum over rows of dy sh: r and two products, then the rows that a workgroup walks (256
    workgroups at least, or all rows by four waves above 8192 values), then what is left of at most 1024
    workgroups by 16 threads each."""
    walked = rows // 4 + 1 if dim > 8192 else rows // 256 + 1
    return rms_count(dim) + 2 + walked + 3 + 1024 // 16 + 16
