"""Small programs that use the library as a user's would."""
