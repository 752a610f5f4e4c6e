// What the files of entry points share: the thread's error text and the device
// check (both in api.cpp).
#pragma once

namespace fp8bq {

// Sets the text that fp8bq_last_error() returns; returns `status`.
int entry_fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// FP8BQ_OK if the current device is a gfx950, else the error (with its text).
int entry_device();

}  // namespace fp8bq
