"""Sizes of the 4-bit products by the kernel that they reach. tests/test_mxfp4_choices.py
holds the choice to this list on the CPU, tests/test_gpu_mxfp4_kernels.py runs it: a
changed rule that leaves a kernel without a test is seen at once."""
import torch

import mx4_ref

# how a kernel's mangled name begins; the last for sums of K's parts
SKINNY16, SKINNY32 = "mx4_skinny_kernelILi1E", "mx4_skinny_kernelILi2E"
T64, T128, T256 = "mx4_tile_kernelILi64E", "mx4_tile_kernelILi128E", "mx4_big_kernelE"
SPLIT = "mx4_reduce_kernel"

# m, n, k. 256 x 256: depths of an odd and an even count of runs (of 128) and of stages (of 256), up to
# three groups of four stages' scales and one run over; last tiles of one row and one column up to whole
# ones; N of every alignment
LINEAR = [
    ((T256,), 2945, 2947, 896), ((T256,), 2817, 2817, 1152), ((T256,), 2944, 3200, 1024),
    ((T256,), 2818, 2824, 2176), ((T256,), 2821, 2822, 2304), ((T256,), 2817, 2818, 4224),
    ((T128,), 1409, 1535, 1152), ((T128,), 2049, 1025, 640), ((T128,), 129, 12801, 384),
    ((T64,), 65, 130, 1152), ((T64,), 300, 96, 4224), ((T64,), 33, 5000, 896),
    # K in parts: an odd count of runs, parts of unequal length, sums of any alignment
    ((T64, SPLIT), 129, 257, 8320), ((T64, SPLIT), 17, 5000, 8320), ((T64, SPLIT), 70, 101, 12416),
    ((T64, SPLIT), 200, 64, 12416),
    # up to 32 rows: one to eight waves a column set, with a turn that only some of them take
    ((SKINNY32,), 17, 41, 128), ((SKINNY32,), 31, 4096, 1152), ((SKINNY32,), 32, 41, 2688), ((SKINNY32,), 18, 999, 5120),
    ((SKINNY32,), 25, 66, 13824),
    ((SKINNY16,), 16, 41, 1152), ((SKINNY16,), 9, 5001, 2688), ((SKINNY16,), 1, 97, 13824), ((SKINNY16,), 5, 6, 8320),
]

_UNEVEN = [0, 1, 31, 160, 162, 162, 471, 640, 797]
_MANY = [0] + torch.randint(0, 21, (127,), generator=torch.Generator().manual_seed(3)).cumsum(0).tolist() + [1400]
# rows, offsets, n, k
GROUPED = [
    ((T256,), 4100, [3, 4, 1300, 4098], 2100, 384),   # a group of one row, rows before and behind
    ((T256,), 4096, [0, 3839, 4096], 2101, 256),      # one stage
    ((T256,), 4200, [0, 0, 4200], 2049, 1152),        # all rows in one of two
    ((T256,), 4400, [0, 300, 556, 1324, 4399], 2120, 2176),
    ((T128,), 800, _UNEVEN, 2050, 640), ((T128,), 799, _UNEVEN, 2049, 896), ((T128,), 3000, [5, 1000, 1129, 3000], 1031, 1152),
    # few rows a group: many groups with many columns, few with few
    ((T128,), 1400, _MANY, 520, 384), ((T128,), 1400, _MANY, 513, 1152), ((T64,), 1400, _MANY, 512, 384),
    ((T64,), 100, [0, 64, 64, 65, 67, 90, 90, 99, 100], 130, 1152), ((T64,), 800, _UNEVEN, 257, 2176),
    # few rows a group, some with more than a unit of 32
    ((SKINNY32,), 41, [0, 1, 34, 34, 36, 36, 40, 41], 41, 1152), ((SKINNY32,), 42, [0, 1, 34, 34, 36, 36, 40, 41], 300, 2688),
    ((SKINNY32,), 48, [2, 42, 42, 42, 43, 43, 43, 43, 45], 66, 5120), ((SKINNY32,), 30, [0, 17, 17, 18, 18, 30], 41, 13824),
    ((SKINNY32,), 64, [0] * 63 + [33, 64], 97, 384),
]

# m, n, k of the layer; which: 1 dX, 2 dW, 3 both; launches in order (dW first)
BACKWARD = [
    ((T256,), 2945, 2945, 2947, 3),                   # both in one launch
    ((T256,), 2945, 2945, 2947, 1), ((T256,), 2945, 2945, 2947, 2),
    ((T128,), 1200, 1290, 1410, 3), ((T64,), 200, 300, 130, 3),
    # apart, as dX (dW) is deep for a kernel that is not its own
    ((T128, SKINNY32), 20, 12000, 333, 3), ((T64, SKINNY16), 16, 13824, 64, 3), ((SKINNY16, T64), 4000, 16, 320, 3),
    ((T128, T64), 128, 7680, 1024, 3),
    ((T64,), 16, 2048, 640, 3), ((T128,), 128, 2048, 1024, 3),  # in one launch, as neither is
    ((SKINNY32,), 20, 12000, 333, 1), ((T64, SPLIT), 200, 9001, 130, 1), ((T64, SPLIT), 9001, 200, 130, 2),
    ((T64,), 70, 300, 130, 2), ((SKINNY16,), 9, 700, 333, 1),
]

# rows, offsets, n, k of the layer, which
GROUPED_BACKWARD = [
    ((T256, T128), 1540, [2, 2, 700, 1540], 2400, 2403, 3),  # an empty group, odd and even runs
    ((T256,), 4200, [7, 1400, 4150], 2900, 2901, 3),  # both in one launch
    ((T256,), 1100, [0, 100, 1100], 2900, 2818, 2),   # a group of one run
    ((T128,), 800, _UNEVEN, 1031, 2049, 3), ((T128,), 800, _UNEVEN, 1031, 2049, 1),
    ((T128,), 800, _UNEVEN, 640, 650, 2), ((T64,), 300, [0, 200, 200, 299], 130, 70, 2),
    ((T64,), 300, [0, 200, 200, 299], 130, 70, 1),
    ((T128, SKINNY32), 30, [0, 17, 17, 18, 18, 30], 5000, 41, 3), ((T64,), 30, [0, 17, 17, 18, 18, 30], 600, 300, 3),
    ((SKINNY32,), 30, [0, 17, 17, 18, 18, 30], 5000, 41, 1),
]


def case_ids(cases):
    return ["-".join(str(v) for v in (*c[0], *(v if not isinstance(v, list) else f"{len(v) - 1}groups" for v in c[1:])))
            for c in cases]


def rounded(x):
    """float64 values of x [rows][k], finite, in the format: what mx4_ref's codes and scales stand for, by rounding
    to the step between magnitudes (ties to the even multiple, whose code is the even one)."""
    rows, k = x.shape
    v = torch.zeros((rows, mx4_ref.up128(k)), dtype=torch.float64)
    v[:, :k] = x
    v = v.reshape(rows, -1, 32)
    f, e = torch.frexp(v.abs().amax(2, keepdim=True))
    s = torch.exp2((e - 3 + (f > 0.75).int()).clamp(min=-127).double())
    a = v / s
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0)).double()
    return (torch.round(a / step) * step * s).reshape(rows, -1)
