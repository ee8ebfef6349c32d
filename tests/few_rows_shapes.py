"""Shapes of the e4m3 product's few-rows kernel."""

# (t, k, n, experts, experts with rows -> rows), searched for their runs: at the first and the last
# expert, on either side of each 64 and 512 of them, one run of all rows, several in one 64
SCATTERED = [(8, 4112, 4100, 256, {0: 1, 3: 1, 63: 1, 64: 1, 65: 1, 127: 1, 200: 1, 255: 1}),
             (8, 1040, 513, 256, {255: 8}), (4, 2048, 1040, 64, {0: 1, 31: 2, 63: 1}),
             (20, 4112, 48, 4096, {0: 3, 511: 1, 512: 1, 513: 2, 1023: 1, 1024: 4, 3583: 1, 3584: 2, 4095: 5}),
             (12, 2064, 1008, 1000, {448: 1, 449: 1, 511: 1, 999: 1}), (6, 2064, 2000, 700, {600: 5, 699: 1}),
             (3, 2048, 600, 513, {512: 3}), (5, 1040, 640, 512, {511: 4}), (7, 2064, 1008, 300, {})]

# Rows of each expert (None: one matrix), k, n; whether in passes of 16 rows or of 64.  Experts of more
# rows than a pass, K steps of a wave that end with one and with two in flight, K ends of 16 to 112.
PASSES = [(None, 1, 8192, 8192, 16), (None, 3, 14352, 4096, 16), (None, 16, 4208, 1030, 16), (None, 2, 1136, 48, 16),
          (None, 65, 2048, 96, 64), (None, 17, 2176, 1000, 64), (None, 33, 3200, 96, 64), (None, 24, 7280, 4096, 64),
          ([17, 0, 1, 33, 0, 60, 0, 2] + [0] * 40, 4176, 132, 16), ([40] + [0] * 12, 2048, 1030, 16),
          ([3, 1, 0, 29, 0, 0, 7, 16] + [0] * 9, 7184, 520, 16), ([0] * 31 + [128], 1296, 36, 16),
          ([65, 1, 130, 0, 20, 33, 7], 4112, 100, 64), ([0, 0, 200, 5], 5168, 48, 64), ([40, 9, 64, 16, 17], 16384, 80, 64)]

# Calls of up to 16 rows: (t, k, n, rows of each expert or None)
SIXTEEN = [(1, 16, 8, None), (1, 256, 4096, None), (2, 144, 33, None), (16, 256, 512, None), (7, 400, 1001, None),
           (2, 5120, 16384, None), (16, 2048, 16384, None), (1, 7168, 16384, None), (16, 8192, 8192, None),
           (12, 16384, 1000, None), (8, 256, 512, [1] * 8), (8, 272, 1040, [0, 3, 0, 5]), (16, 2048, 4096, [0, 16, 0, 0]),
           (5, 144, 2000, [0] * 250 + [2, 0, 3]), (16, 512, 48, [0, 0, 9, 1])]

# The same for passes of 64: (t, k, n, rows of each expert or None)
SIXTY_FOUR = [(shape[1], *shape[2:4], None) if shape[0] is None else (sum(shape[0]), *shape[1:3], shape[0])
              for shape in PASSES if shape[-1] == 64]
