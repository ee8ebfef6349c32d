"""Shapes of the e4m3 product's few-rows kernel."""

# (t, k, n, experts, experts with rows -> rows), searched for their runs: at the first and the last
# expert, on either side of each 64 and 512 of them, one run of all rows, several in one 64
SCATTERED = [(8, 4112, 4100, 256, {0: 1, 3: 1, 63: 1, 64: 1, 65: 1, 127: 1, 200: 1, 255: 1}),
             (8, 1040, 513, 256, {255: 8}), (4, 2048, 1040, 64, {0: 1, 31: 2, 63: 1}),
             (20, 4112, 48, 4096, {0: 3, 511: 1, 512: 1, 513: 2, 1023: 1, 1024: 4, 3583: 1, 3584: 2, 4095: 5}),
             (12, 2064, 1008, 1000, {448: 1, 449: 1, 511: 1, 999: 1}), (6, 2064, 2000, 700, {600: 5, 699: 1}),
             (3, 2048, 600, 513, {512: 3}), (5, 1040, 640, 512, {511: 4}), (7, 2064, 1008, 300, {})]
