"""Sizes that take every form of the few-row kernel of the products grouped by
expert, and the form that the launch has to choose: shared by the GPU test
that runs them and the CPU test that asks the planner."""
import random

F32, BF16 = 0, 1

# rows, experts, out, in, dtype, (tiles of rows, K a multiple of a step), rows of some experts
FEW = [
    (384, 64, 264, 128, BF16, (2, 1), [70, 20, 16, 17, 33]),
    (384, 64, 264, 72, BF16, (2, 0), [32, 31, 1]),
    (500, 64, 257, 96, BF16, (2, 1), [65, 15, 30]),
    (500, 64, 273, 130, BF16, (2, 0), [129, 17]),
    (700, 64, 520, 1056, BF16, (2, 1), [40, 18, 16]),
    (700, 70, 263, 2050, BF16, (2, 0), [35, 32, 24]),
    (200, 64, 256, 32, BF16, (2, 1), [60, 17]),
    (900, 130, 130, 40, BF16, (2, 0), [100, 20]),
    (13, 6, 2750, 64, BF16, (2, 1), [12]),
    (64, 2, 8192, 48, BF16, (2, 0), [40]),
    (24, 1, 16390, 33, BF16, (2, 0), []),
    (300, 65, 270, 5, BF16, (2, 0), [66, 18]),
    (300, 65, 270, 1, BF16, (2, 0), [17]),
    (384, 64, 264, 128, F32, (2, 1), [70, 20, 16, 17, 33]),
    (1500, 64, 264, 75, F32, (2, 0), [100, 31, 1]),
    (500, 64, 257, 48, F32, (2, 1), [65, 15, 30]),
    (500, 64, 273, 65, F32, (2, 0), [129, 17]),
    (900, 130, 128, 528, F32, (2, 1), [40, 18, 16]),
    (24, 1, 16390, 33, F32, (2, 0), []),
    (300, 65, 270, 3, F32, (2, 0), [66, 18]),
    (300, 65, 270, 1, F32, (2, 0), [17]),
    (9, 4, 40, 64, BF16, (1, 1), [7]),
    (9, 4, 41, 70, BF16, (1, 0), []),
    (9, 4, 40, 48, F32, (1, 1), [7]),
    (9, 4, 41, 50, F32, (1, 0), []),
    (64, 4, 72, 96, BF16, (4, 1), []),
    (60, 4, 71, 97, BF16, (4, 0), [57]),
    (96, 4, 72, 96, F32, (4, 1), [66]),
    (60, 4, 71, 97, F32, (4, 0), []),
]


def counts(case):
    """Rows of every expert: those the case names, at random places, the rest
    spread over the others, of which some stay without."""
    rows, experts, *_, some = case
    rng = random.Random(rows * 31 + experts)
    n = [0] * experts
    places = rng.sample(range(experts), len(some))
    for p, k in zip(places, some):
        n[p] = k
    rest = [e for e in range(experts) if e not in places] or [0]
    rest = rng.sample(rest, max(1, len(rest) * 4 // 5))
    for _ in range(rows - sum(some)):
        n[rng.choice(rest)] += 1
    return n

# Products that take the large tiles: pass, rows, experts, out, in
FORWARD, WEIGHT, INPUT = 0, 1, 2
LARGE = [
    (FORWARD, 9000, 12, 5125, 1288), (FORWARD, 20000, 30, 1157, 264), (FORWARD, 30000, 9, 513, 72),
    (FORWARD, 9000, 12, 5128, 1288), (INPUT, 9000, 12, 5128, 1288), (WEIGHT, 9000, 12, 5128, 1288),
    (FORWARD, 20000, 30, 1160, 2056), (INPUT, 20000, 30, 1160, 2056), (WEIGHT, 20000, 30, 1160, 2056),
    (FORWARD, 5000, 3, 5128, 5144), (INPUT, 5000, 3, 5128, 5144), (WEIGHT, 5000, 3, 5128, 5144),
]
