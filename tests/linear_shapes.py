"""Sizes at which the linear layer's products take each of its tiles, for the GPU tests to run and for
the CPU tests to hold against the plan: a refitted plan that moves one of them fails there.

A product's order is "fwd" (x W^T: rows m, columns n, over k), "dx" (dz W: m, k, over n) or "dw" (dz^T x: n, k, over m). Each
size is (m, k, n) with k = 2 mod 8 and odd m and n; n + 1 takes the same tile and split. The shape
numbers are those of zero_gemm_plan.h."""

# (order, shape, k split over blocks): size
TILES = {
    ("fwd", 0, False): (8147, 202, 1345),
    ("fwd", 1, False): (3661, 1410, 843),
    ("fwd", 1, True): (1861, 4066, 453),
    ("fwd", 2, False): (5421, 170, 1409),
    ("fwd", 2, True): (387, 5506, 5449),
    ("fwd", 3, True): (73, 5130, 3531),
    ("fwd", 4, False): (33, 154, 9),
    ("fwd", 4, True): (33, 1154, 9),
    ("fwd", 5, False): (6003, 834, 1281),
    ("fwd", 5, True): (7369, 5834, 257),
    ("fwd", 6, False): (7207, 154, 1027),
    ("fwd", 6, True): (7825, 5914, 387),
    ("fwd", 7, False): (37, 194, 7),
    ("fwd", 7, True): (309, 1730, 97),
    ("dx", 0, False): (2317, 4938, 151),
    ("dx", 0, True): (1541, 2506, 8207),
    ("dx", 1, False): (1539, 3290, 151),
    ("dx", 1, True): (601, 1474, 4067),
    ("dx", 2, False): (1411, 5418, 151),
    ("dx", 2, True): (409, 5538, 5517),
    ("dx", 3, True): (67, 3522, 5141),
    ("dx", 4, False): (33, 10, 151),
    ("dx", 4, True): (33, 10, 1153),
    ("dx", 5, False): (2881, 3914, 153),
    ("dx", 5, True): (897, 2818, 6793),
    ("dx", 6, False): (1665, 4642, 155),
    ("dx", 6, True): (899, 2714, 6801),
    ("dx", 7, False): (33, 10, 193),
    ("dx", 7, True): (33, 10, 6145),
    ("dw", 0, False): (163, 4874, 2313),
    ("dw", 0, True): (8237, 5418, 645),
    ("dw", 1, False): (153, 5914, 833),
    ("dw", 1, True): (4145, 3450, 195),
    ("dw", 2, False): (167, 5378, 1413),
    ("dw", 2, True): (6429, 5258, 135),
    ("dw", 3, True): (2305, 4810, 9),
    ("dw", 4, False): (151, 10, 9),
    ("dw", 4, True): (1187, 10, 7),
    ("dw", 5, False): (155, 5914, 1923),
    ("dw", 5, True): (6341, 5522, 389),
    ("dw", 6, False): (151, 4618, 1679),
    ("dw", 6, True): (6639, 4410, 513),
    ("dw", 7, False): (193, 10, 9),
    ("dw", 7, True): (6145, 10, 9),
}
CANDIDATES = range(8)
STAND_IN = 8

# forward (m, k, n) whose planned small tiles are more than a grid holds
TOO_MANY_TILES = (108_003_333, 8, 258)


def product(order, m, k, n):
    """(rows, columns, k) of the product of that order in a layer of m tokens, k features in, n out."""
    return {"fwd": (m, n, k), "dx": (m, k, n), "dw": (n, k, m)}[order]
